"""Calls of the binding on a stream that is not the current one, with temporaries of their own."""
import pytest
import torch

from block_sparse_video_rearrange_b200 import rf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("span", ["row", "sample"])
def test_group_norm_on_a_side_stream_keeps_its_temporaries(span, raw):
    """The kernels start only after the call has returned and the current stream has allocated, and written, memory of
    the sizes of the call's temporaries: they must not be the same memory."""
    gen = torch.Generator().manual_seed(6)
    x, dy = (torch.randn(2, 500, 3, 40, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    gamma, beta = (torch.randn(3, 40, generator=gen).cuda() for _ in range(2))
    stats = rf.group_norm_stats(x, span)
    want = [torch.empty_like(t) for t in (x, x, gamma, beta)]
    rf.group_norm(x, gamma, beta, want[0], span=span, act="silu", stats=stats)
    rf.group_norm_backward(x, gamma, beta, dy, stats, *want[1:], span=span, act="silu")
    got = [torch.empty_like(t) for t in want]
    sizes = [rf.group_norm_workspace(x, span).numel(), 2 * 3 * 2]
    side = torch.cuda.Stream()

    def junk():
        return [torch.full((n,), 2 ** 30 + 12345, dtype=torch.int32, device="cuda") for n in sizes * 20]
    junk()                                                # the memory is in the pool, the kernel loaded
    torch.cuda.synchronize()
    for call in (lambda s: rf.group_norm(x, gamma, beta, got[0], span=span, act="silu", stream=s),
                 lambda s: rf.group_norm_backward(x, gamma, beta, dy, stats, *got[1:], span=span, act="silu", stream=s)):
        waited = False
        for _ in range(3):                                # a busy host may be slower than the sleep
            with torch.cuda.stream(side):
                torch.cuda._sleep(400_000_000)            # some 200 ms before the kernels can start
            call(side.cuda_stream if raw else side)
            taken = junk()
            torch.cuda.current_stream().synchronize()     # written while the side stream still waits
            waited = waited or not side.query()
            torch.cuda.synchronize()
            del taken
            if waited:
                break
        assert waited
    for a, b in zip(got, want):
        assert torch.equal(a, b)
