"""The bounded waits of the shared-prefix decode's two pipelined kernels, made to run out on purpose: the status word
and the roles say so, nothing hangs, and the next call is right bit for bit."""
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

from shared_prefix_checks import DEV, Case
from test_gpu_rope_q4 import _lib  # noqa: F401  (builds and loads the library)

pytestmark = pytest.mark.gpu
LIMIT_NS = 20_000_000


@pytest.fixture(autouse=True)
def _normal_waits_after():
    yield
    pa.set_wait_test()


@pytest.fixture(scope="module")
def case():
    # 96 sequences of up to 900 own tokens over 8192 shared ones: both kernels' CTAs pass the stall points and rings
    c = Case([(96, 8192)], [900, 700, 333, 800], 32, 8, 128, 16, torch.bfloat16, seed=1)
    return c, c.run().clone()


@pytest.mark.parametrize("stall,sites,none", [
    (pa.STALL_NONE, [], 31),
    (pa.STALL_PRODUCER, [pa.WAIT_DECODE_CONSUMER, pa.WAIT_PREFILL_MMA, pa.WAIT_PREFILL_SOFTMAX],
     pa.WAIT_DECODE_PRODUCER | pa.WAIT_PREFILL_PRODUCER),
    (pa.STALL_CONSUMER, [pa.WAIT_DECODE_PRODUCER, pa.WAIT_PREFILL_PRODUCER, pa.WAIT_PREFILL_SOFTMAX],
     pa.WAIT_DECODE_CONSUMER | pa.WAIT_PREFILL_MMA)])
def test_waits_that_run_out(case, stall, sites, none):
    c, want = case
    status, seen = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in "ab")
    pa.set_wait_test(LIMIT_NS, stall, 3, seen)
    out = c.run(dev_status=status)
    torch.cuda.synchronize()
    pa.set_wait_test()
    got = int(seen.item())
    assert all(got & s for s in sites) and not got & none, hex(got)
    assert pa.get_device_status(status) == (pa.OK if stall == pa.STALL_NONE else pa.ERR_TIMEOUT)
    if stall == pa.STALL_NONE:
        assert torch.equal(out, want)
    status.zero_()
    assert torch.equal(c.run(dev_status=status), want)
    assert pa.get_device_status(status) == pa.OK
