"""States of the selective scan at addresses that are no multiple of 16 bytes: refused where the states of a channel
are whole fours, which kernels move at once; elsewhere any slice of a pool serves."""
import pytest
import torch

from tests.test_scan_api import FAKE, INV, L, P, run_scan, scan, scan_back, scan_step


def test_whole_fours_need_16_bytes_and_others_an_element():
    for n, off in ((16, 4), (16, 8), (4, 12), (5, 2), (5, 1), (1, 3)):
        d = scan(n=n)
        for st in (run_scan(d, s0=P[5] + off), run_scan(d, s1=P[5] + off), scan_back(d, s0=P[5] + off), scan_back(d, ds0=P[5] + off),
                   scan_back(d, ds1=P[5] + off), scan_step(scan(n=n, N=1), state=FAKE + off)):
            assert st == INV and b"aligned" in L.rn_last_error(), (n, off)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 5, 21])
def test_slices_of_a_pool(n):
    import linear_recurrent_sequence_rn_amd as rn
    S, N, D, dev = 3, 100, 7, "cuda:0"
    g = torch.Generator().manual_seed(n)
    r = lambda *s: torch.randn(*s, generator=g).to(dev)  # noqa: E731
    x, dt, dy, A, B, C = r(S, N, D), r(S, N, D), r(S, N, D), -r(D, n).abs(), r(S, 1, N, n), r(S, 1, N, n)
    pool = r(8, D, n)
    whole, cut = pool[1:4].clone(), pool[1:4]
    assert cut.data_ptr() % 16
    want, last = rn.rn_selective_scan_chunked(x, dt, A, B, C, state_in=whole, state_out=True)
    out, state = rn.rn_selective_scan_chunked(x, dt, A, B, C, state_in=cut, state_out=pool[5:8])
    assert torch.equal(out, want) and torch.equal(state, last)
    a = rn.rn_selective_scan_backward(dy, x, dt, A, B, C, state_in=whole, dstate_out=last.clone(), want_dstate_in=True)
    b = rn.rn_selective_scan_backward(dy, x, dt, A, B, C, state_in=cut, dstate_out=pool[5:8], want_dstate_in=True)
    assert all(torch.equal(a[k], b[k]) for k in a)
    one = lambda t: t[..., :1, :]  # noqa: E731
    want = rn.rn_selective_scan_step(one(x), one(dt), A, one(B), one(C), whole)
    assert torch.equal(rn.rn_selective_scan_step(one(x), one(dt), A, one(B), one(C), cut), want) and torch.equal(cut, whole)
