"""More host-side refusals of the gated rule's C entry points (no GPU: nothing is launched)."""
import ctypes

from test_gated_abi import P, lib, shape  # noqa: F401


def test_states_do_not_lie_over_the_offsets(lib):  # noqa: F811
    """A state written over the packed offsets that other CTAs still read; the state in place of S0 is fine
    (a refused workspace proves that the aliasing checks passed: it comes last)."""
    s = shape(packed=True)
    for S0, Sf, want in ((None, P[8], 1), (P[8], P[8], 1), (None, P[8] - 2 * 4 * 64 * 32 * 4, 4), (P[9], P[9], 4)):
        rc = lib.efla_gated_fwd(ctypes.byref(s), P[8], *P[:5], S0, P[5], Sf, None, 0, None)
        assert rc == want and lib.efla_last_error().decode()
