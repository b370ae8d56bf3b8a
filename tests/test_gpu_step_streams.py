"""The end-to-end step on a stream that is not the current one."""
import numpy as np
import pytest
import torch

from helpers import golden_workload
from helpers_kv8 import bits
from tree_verification_jsv_b200 import jsv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("kind", ["VerifyStep", "VerifyStepKv8"])
def test_run_host_keeps_its_copies_on_the_stream_it_is_given(kind, raw):
    """With the current stream held up for a tenth of a second, the step on
    another stream still takes the inputs that were written for it, and its
    results are there when that stream is done."""
    from tree_verification_jsv_b200 import step
    wl, tokens, _ = golden_workload("tiny")
    st = getattr(step, kind)(wl, tokens)
    q = st.host_inputs()["q"]
    first = q.clone()
    caches = [(x, x.clone()) for x in (st.k_cache, st.v_cache)]

    def restore():                      # a step moves the accepted path's rows
        for x, y in caches:
            x.copy_(y)
        torch.cuda.synchronize()

    st.run()
    torch.cuda.synchronize()
    want, lens = bits(st.out), {k: v.cpu() for k, v in st._out.dev.items()}
    restore()
    q.copy_(torch.flip(first, [0]))
    st.run_host()
    torch.cuda.synchronize()
    assert not np.array_equal(bits(st.out), want)
    restore()
    q.copy_(first)
    st._out.host_buf.zero_()
    side = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)
    out = st.run_host(side.cuda_stream if raw else side)
    side.synchronize()
    assert all(torch.equal(out[k], v) for k, v in lens.items())
    torch.cuda.synchronize()
    assert np.array_equal(bits(st.out), want) and int(st.status.item()) == 0


@pytest.mark.parametrize("kind", ["VerifyStep", "VerifyStepKv8"])
def test_run_host_on_the_default_stream_by_its_handle(kind):
    from tree_verification_jsv_b200 import step
    wl, tokens, _ = golden_workload("tiny")
    st = getattr(step, kind)(wl, tokens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        out = st.run_host(0)
        torch.cuda.default_stream().synchronize()
        assert not side.query()                     # nothing of the step waited for it
    got = {k: v.clone() for k, v in out.items()}
    torch.cuda.synchronize()
    assert all(torch.equal(v, getattr(st, k).cpu()) for k, v in got.items()) and int(st.status.item()) == 0
