"""Sizes of the convolution's, the scan's and the RMS norm's calls past 32 bits.  Stand-ins for tensors and the library: no GPU
needed, nothing is launched."""
import pytest
import torch

import exact_flow_recurrence_gb300 as efla
from test_devices import F32, Fake, I32, gpus  # noqa: F401

BIG = (1 << 32) + 4     # (its lowest 32 bits are a size that the call would take)


def big_calls():
    w, b = Fake(1, 4, dtype=F32), Fake(1, dtype=F32)
    yield lambda: efla.efla_conv_fwd(Fake(1, BIG, 1), w, b, y=Fake(1, BIG, 1), want_state=False)
    yield lambda: efla.efla_conv_fwd(Fake(8, 1), w, b, offsets=Fake(BIG + 1, dtype=I32), y=Fake(8, 1), S_final=Fake(BIG, 3, 1))
    yield lambda: efla.efla_conv_fwd(Fake(1, 8, 4), Fake(4, BIG, dtype=F32), y=Fake(1, 8, 4), want_state=False)
    yield lambda: efla.efla_conv_step(Fake(BIG, 1), w, Fake(8, 3, 1), slots=Fake(BIG, dtype=I32), y=Fake(BIG, 1))
    yield lambda: efla.efla_conv_step(Fake(2, 1), w, Fake(BIG, 3, 1), y=Fake(2, 1))
    scan = lambda L, D, G, N: (Fake(1, L, D), Fake(1, L, D), Fake(D, N, dtype=F32), Fake(1, L, G, N), Fake(1, L, G, N))  # noqa: E731
    for L, D, G, N in ((BIG, 1, 1, 1), (8, BIG, 1, 1), (8, 4, BIG, 1), (8, 4, 1, BIG)):
        yield lambda a=scan(L, D, G, N): efla.efla_scan_fwd(*a, y=Fake(*a[0].shape), want_state=False, workspace=Fake(1 << 20, dtype=torch.uint8))
    one = (Fake(2, 1), Fake(2, 1), Fake(1, 4, dtype=F32), Fake(2, 1, 4), Fake(2, 1, 4))
    yield lambda: efla.efla_scan_step(*one, Fake(BIG, 1, 4, dtype=F32), y=Fake(2, 1))
    yield lambda: efla.efla_rms_fwd(Fake(4, 256), Fake(256, dtype=F32), group=1 << 32, y=Fake(4, 256, dtype=torch.float8_e4m3fn),
                                    scale=Fake(4, 1, dtype=F32), rstd=Fake(4, dtype=F32))
    yield lambda: efla.efla_rms_fwd(Fake(2, BIG), Fake(BIG, dtype=F32), y=Fake(2, BIG), rstd=Fake(2, dtype=F32))


@pytest.mark.parametrize("call", list(big_calls()))
def test_sizes_past_32_bits_are_refused(gpus, call):  # noqa: F811
    """The C structs hold 32 bits: a longer size is refused, not cut."""
    with pytest.raises(ValueError, match="2\\^31"):
        call()
    assert gpus.seen == []
