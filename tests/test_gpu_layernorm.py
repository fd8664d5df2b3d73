"""Layer norm and its gradients on the GPU against the float64 oracle.

Tolerances. u = 2^-24. Sums over a row run over at most 64 values a lane and 10 joins, so the
mean is off by at most 74 u mean|h| and the variance, relatively, by at most 80 u (plus the
square of the mean's error): the normalised value xh by at most 80 u (rms(h) rstd + |xh|),
counting the roundings around. A result in bf16 adds half a step, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from oracle import block as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rn():
    import linear_recurrent_sequence_rn_amd as m
    return m


def half_step(t):
    return torch.finfo(t).eps / 2


def np64(t):
    return t.detach().double().cpu().numpy()


def rows(gen, n, d, dt, mean=0.25, std=1.5):
    return (torch.randn(n, d, generator=gen) * std + mean).to(dt)


def spread(gen, n, d, dt, extra):
    """A [n, d] view of a wider buffer: rows `extra` elements apart from each other."""
    wide = torch.zeros(n, d + extra, dtype=dt, device=DEV)
    wide[:, :d] = rows(gen, n, d, dt).to(DEV)
    return wide[:, :d]


def check(got, want, tol):
    off = np.abs(np64(got) - want)
    assert (off <= tol).all(), f"{(off / tol).max()} of the tolerance"


SIZES = [(1, 1), (3, 2), (5, 7), (1, 64), (4, 512), (9, 513), (2, 1024), (130, 1000), (33, 1537), (7, 2048),
         (5, 2056), (3, 4096), (6, 4100), (2, 8192), (3, 8200), (2, 16384), (2, 16383), (2049 * 4 + 1, 64), (2100, 2560)]


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16->f32", "f32->bf16"])
def test_forward(n, d, kind):
    dt, od = DT[kind.split("->")[0]], DT[kind.split("->")[-1]]
    g = torch.Generator().manual_seed(n * 31 + d)
    x, r = rows(g, n, d, dt), rows(g, n, d, dt, 0.0, 1.0)
    w, b = torch.randn(d, generator=g) * 0.2 + 1, torch.randn(d, generator=g) * 0.2
    for res, aff in ((None, True), (r, False), (r, True)):
        y, h = K.layernorm(x, w if aff else None, b if aff else None, 1e-5, res)
        xh, _ = K.layernorm(x, None, None, 1e-5, res)
        got = rn().rn_layernorm(x.to(DEV), w.to(DEV) if aff else None, b.to(DEV) if aff else None,
                                residual=None if res is None else res.to(DEV), out_dtype=od)
        out, total = got if res is not None else (got, None)
        assert out.dtype == od and out.shape == (n, d)
        rms = np.sqrt((h * h).mean(-1, keepdims=True) / (h.var(-1, keepdims=True) + 1e-5))
        ww, bb = (np64(w), np64(b)) if aff else (1.0, 0.0)
        check(out, y, 80 * U * (rms + np.abs(xh)) * np.abs(ww) + 2 * U * np.abs(bb) + half_step(od) * 1.01 * np.abs(y) + 1e-30)
        if res is not None:
            assert total.dtype == dt
            check(total, h, (U + half_step(dt)) * 1.01 * np.abs(h))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("d,extra", [(256, 8), (256, 1), (100, 28), (4096, 4096)])
def test_strided_rows_and_in_place(kind, d, extra):
    dt = DT[kind]
    g = torch.Generator().manual_seed(d + extra)
    x, r = spread(g, 37, d, dt, extra), spread(g, 37, d, dt, 2 * extra)
    base = x._base
    y, h = K.layernorm(x.cpu(), None, None, 1e-5, r.cpu())
    want, total = rn().rn_layernorm(x, residual=r)
    keep_r = r.clone()
    out, s = rn().rn_layernorm(x, residual=r, out=x, sum_out=r)        # both in place
    assert out is x and s is r
    assert torch.equal(out, want) and torch.equal(s, total) and not torch.equal(keep_r, r)
    assert int(torch.count_nonzero(base[:, d:])) == 0                  # nothing between the rows
    check(out, y, 80 * U * (np.sqrt((h * h).mean(-1, keepdims=True)) / h.std(-1, keepdims=True) + np.abs(y))
          + half_step(dt) * 1.01 * np.abs(y))
    # an input whose rows are all the same row
    one = rows(g, 1, d, dt).to(DEV)
    same = rn().rn_layernorm(one.expand(5, d))
    assert torch.equal(same, rn().rn_layernorm(one).expand(5, d))
    # leading axes that step like one, and ones that do not
    z = torch.zeros(4, 6, d + extra, dtype=dt, device=DEV)[..., :d]
    assert rn().rn_layernorm(z).shape == z.shape
    with pytest.raises(ValueError):
        rn().rn_layernorm(z.transpose(0, 1))


def test_eps_zero_constant_and_nonfinite_rows():
    x = torch.full((6, 96), 3.0, device=DEV)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[4] = torch.arange(96.0)
    w, b = torch.full((96,), 2.0, device=DEV), torch.full((96,), -1.0, device=DEV)
    out = rn().rn_layernorm(x, w, b)
    assert torch.equal(out[0], b) and torch.equal(out[3], b) and torch.equal(out[5], b)
    assert out[1].isnan().all() and out[2].isnan().all()
    assert out[4].isfinite().all()
    assert rn().rn_layernorm(x[:1], w, b, 0.0).isnan().all()           # 0 / 0
    assert torch.equal(rn().rn_layernorm(x[4:5], w, b), out[4:5])      # rows do not meet


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16->f32"])
def test_backward(n, d, kind):
    """dx: two further means of products of sizes |g| and |g xh|, and xh's own error; sums over
    rows: at most n/1024 + 5 rows one after another, 32 + 16 joins of partial sums, each term
    with xh's error."""
    dt, od = DT[kind.split("->")[0]], DT[kind.split("->")[-1]]
    g = torch.Generator().manual_seed(n * 17 + d)
    x, dy, dh = rows(g, n, d, dt), rows(g, n, d, od, 0.1, 1.0), rows(g, n, d, dt, 0.0, 1.0)
    w = torch.randn(d, generator=g) * 0.2 + 1
    for res, aff in ((None, True), (dh, False), (dh, True)):
        ww = w if aff else None
        dx, dw, db = K.layernorm_backward(dy, x, ww, 1e-5, res)
        got = rn().rn_layernorm_backward(dy.to(DEV), x.to(DEV), None if ww is None else ww.to(DEV),
                                         dsum=None if res is None else res.to(DEV))
        xx, gg = np64(x), np64(dy) * (np64(w) if aff else 1.0)
        sd = np.sqrt(xx.var(-1, keepdims=True) + 1e-5)
        xh = (xx - xx.mean(-1, keepdims=True)) / sd
        exh = 80 * U * (np.sqrt((xx * xx).mean(-1, keepdims=True)) / sd + np.abs(xh))
        m1, m2 = np.abs(gg).mean(-1, keepdims=True), np.abs(gg * xh).mean(-1, keepdims=True)
        e2 = (np.abs(gg) * exh).mean(-1, keepdims=True) + 80 * U * m2
        tol = (90 * U * (np.abs(gg) + m1 + np.abs(xh) * m2) + exh * m2 + np.abs(xh) * e2) / sd
        tol = tol + half_step(dt) * 1.01 * np.abs(dx) + (0 if res is None else U * np.abs(np64(res)))
        check(got["dx"], dx, tol + 1e-30)
        chain = n / 1024 + 5 + 48
        check(got["dweight"], dw, (np.abs(np64(dy)) * (exh + chain * U * np.abs(xh))).sum(0) + 1e-30)
        check(got["dbias"], db, chain * U * np.abs(np64(dy)).sum(0) + 1e-30)
        assert got["dx"].dtype == dt and got["dweight"].dtype == got["dbias"].dtype == torch.float32


def test_backward_against_differences():
    """The float32 forward call's own differences: (f(x + e) - f(x - e)) / 2e of loss =
    sum(dy y) + sum(dh h) at e = 2^-6: the truncation error is of order e^2, the rounding error
    of y, 1e-6 a value, over e."""
    g = torch.Generator().manual_seed(5)
    x, dy, dh = (torch.randn(3, 40, generator=g).to(DEV) for _ in range(3))
    w, b = (torch.randn(40, generator=g) * 0.3 + 1).to(DEV), torch.randn(40, generator=g).to(DEV)
    got = rn().rn_layernorm_backward(dy, x, w, dsum=dh)

    def loss(x_, w_, b_):
        y, s = rn().rn_layernorm(x_, w_, b_, sum_out=torch.empty_like(x_))
        return ((y.double() * dy).sum() + (s.double() * dh).sum()).item()

    e = 2.0 ** -6
    for a, grad, f in ((x, got["dx"], lambda t: loss(t, w, b)), (w, got["dweight"], lambda t: loss(x, t, b)),
                       (b, got["dbias"], lambda t: loss(x, w, t))):
        flat = grad.flatten()
        for i in range(0, a.numel(), 7):
            up, dn = a.clone(), a.clone()
            up.view(-1)[i] += e
            dn.view(-1)[i] -= e
            num = (f(up) - f(dn)) / (2 * e)
            assert abs(num - flat[i].item()) < 4e-3 * max(1.0, abs(num)), (i, num, flat[i].item())


def test_backward_options():
    g = torch.Generator().manual_seed(6)
    x, dy, dh = (torch.randn(300, 130, generator=g).to(DEV) for _ in range(3))
    w = torch.randn(130, generator=g).to(DEV)
    full = rn().rn_layernorm_backward(dy, x, w, dsum=dh)
    again = rn().rn_layernorm_backward(dy, x, w, dsum=dh)
    assert all(torch.equal(full[k], again[k]) for k in full)           # the same bits
    only = rn().rn_layernorm_backward(dy, x, w, dsum=dh, want_dweight=False, want_dbias=False)
    assert set(only) == {"dx"} and torch.equal(only["dx"], full["dx"])
    one = rn().rn_layernorm_backward(dy, x, w, dsum=dh, want_dbias=False)
    assert torch.equal(one["dweight"], full["dweight"]) and "dbias" not in one
    ws = torch.empty(rn().rn_layernorm_backward_workspace_bytes(dy, x), dtype=torch.uint8, device=DEV)
    ws.fill_(255)
    assert torch.equal(rn().rn_layernorm_backward(dy, x, w, dsum=dh, workspace=ws)["dbias"], full["dbias"])
    with pytest.raises(rn().RnError, match="RN_ERR_WORKSPACE"):
        rn().rn_layernorm_backward(dy, x, w, workspace=ws[:16])
    d2 = dy.clone()
    assert torch.equal(rn().rn_layernorm_backward(d2, x, w, dsum=dh, dx=d2)["dx"], full["dx"])   # over dout
    d3 = dh.clone()
    assert torch.equal(rn().rn_layernorm_backward(dy, x, w, dsum=d3, dx=d3)["dx"], full["dx"])   # over dsum


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("d,extra", [(256, 8), (256, 1), (100, 28), (2000, 3)])
def test_backward_of_strided_rows(kind, d, extra):
    """Rows with gaps, and rows that are all the same one: the bits of the contiguous call where
    the same kernel runs, and its numbers where the rows' alignment takes another."""
    dt = DT[kind]
    g = torch.Generator().manual_seed(d * 3 + extra)
    x, dy, dh, dx = (spread(g, 37, d, dt, n * extra) for n in (1, 2, 3, 4))
    w = torch.randn(d, generator=g).to(DEV)
    got = rn().rn_layernorm_backward(dy, x, w, dsum=dh, dx=dx)
    assert got["dx"] is dx and int(torch.count_nonzero(dx._base[:, d:])) == 0
    want = rn().rn_layernorm_backward(*(t.contiguous() for t in (dy, x)), w, dsum=dh.contiguous())
    for name in ("dx", "dweight", "dbias"):
        a, b = got[name].double(), want[name].double()
        assert (a - b).abs().max() <= (2 * half_step(dt) if name == "dx" else 1e-5) * b.abs().max() + 1e-6
    one = dy[:1].contiguous()
    same = rn().rn_layernorm_backward(one.expand(37, d), x, w)
    full = rn().rn_layernorm_backward(one.expand(37, d).contiguous(), x, w)
    assert all(torch.equal(same[n], full[n]) or extra % 8 for n in full)


def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    for kw in (dict(residual=torch.zeros(4, 65, device=DEV)), dict(residual=x.bfloat16()), dict(weight=x[0].bfloat16()),
               dict(weight=torch.zeros(63, device=DEV)), dict(bias=torch.zeros(64)), dict(out=torch.zeros(3, 64, device=DEV)),
               dict(sum_out=x.bfloat16())):
        with pytest.raises(ValueError):
            rn().rn_layernorm(x, **kw)
    for empty in (torch.zeros(0, 64, device=DEV), torch.zeros(4, 0, device=DEV), torch.tensor(1.0, device=DEV)):
        with pytest.raises(ValueError):
            rn().rn_layernorm(empty)
        with pytest.raises(ValueError):
            rn().rn_layernorm_backward(empty, empty)
    with pytest.raises(TypeError):
        rn().rn_layernorm(x.half())
    with pytest.raises(ValueError):
        rn().rn_layernorm(torch.zeros(64, 4, device=DEV).t())
    with pytest.raises(rn().RnError, match="RN_ERR_UNSUPPORTED"):
        rn().rn_layernorm(torch.zeros(1, 16392, device=DEV))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(40, 64), (9, 1001), (5, 4096), (3, 9003)])
def test_tensors_that_start_at_any_element(kind, n, d):
    """x, residual, weight, bias and the outputs one element into their buffers: the same bits as
    from aligned copies where the pieces are the same, and nothing in front of or behind them."""
    dt = DT[kind]
    g = torch.Generator().manual_seed(d)
    flat = lambda t: torch.cat([t.new_full((1,), 7.0), t.reshape(-1), t.new_full((1,), 7.0)]).to(DEV)  # noqa: E731
    bufs = [flat(rows(g, n, d, dt)) for _ in range(5)]
    x, r, out, total, dy = (b[1:-1].view(n, d) for b in bufs)
    wb = [flat(torch.randn(d, generator=g)) for _ in range(2)]
    w, b = (t[1:-1] for t in wb)
    y, h = K.layernorm(x.cpu(), w.cpu(), b.cpu(), 1e-5, r.cpu())
    xh, _ = K.layernorm(x.cpu(), None, None, 1e-5, r.cpu())
    rn().rn_layernorm(x, w, b, residual=r, out=out, sum_out=total)
    rms = np.sqrt((h * h).mean(-1, keepdims=True) / (h.var(-1, keepdims=True) + 1e-5))
    check(out, y, 80 * U * (rms + np.abs(xh)) * np.abs(np64(w)) + 2 * U * np.abs(np64(b)) + half_step(dt) * 1.01 * np.abs(y) + 1e-30)
    check(total, h, (U + half_step(dt)) * 1.01 * np.abs(h))
    want = rn().rn_layernorm_backward(dy.clone(), total.clone(), w.clone())
    got = rn().rn_layernorm_backward(dy, total, w, dx=x)
    scale = {k: float(v.abs().max()) for k, v in want.items()}
    for k in ("dx", "dweight", "dbias"):     # the two differ in the order of float32 sums and in dx's rounding
        assert float((got[k].float() - want[k].float()).abs().max()) <= (1e-5 + 2 * half_step(got[k].dtype)) * scale[k]
    for t in bufs + wb:
        assert float(t[0]) == 7.0 and float(t[-1]) == 7.0


@pytest.mark.parametrize("n,d", [(1, 17), (15, 64), (1000, 65), (777, 129), (300, 200), (50, 255), (13000, 128), (33, 257)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16->f32"])
def test_narrow_rows(n, d, kind):
    """Rows of a head's width, several to a wave, in numbers that leave waves and blocks part empty."""
    test_forward(n, d, kind)
    test_backward(n, d, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("d,extra", [(256, 8), (256, 1), (100, 28), (2000, 3), (1537, 0)])
def test_backward_of_one_repeated_gradient_row(kind, d, extra):
    """An output gradient that is one row repeated by a stride of 0, beside rows of x with and without
    gaps: alignment takes the same kernel as for the copied rows, and so the same bits come out."""
    g = torch.Generator().manual_seed(d + extra)
    x = spread(g, 37, d, DT[kind], extra)
    one = torch.randn(1, d, generator=g).to(DT[kind]).to(DEV)
    w = torch.randn(d, generator=g).to(DEV)
    same = rn().rn_layernorm_backward(one.expand(37, d), x, w)
    full = rn().rn_layernorm_backward(one.expand(37, d).contiguous(), x, w)
    assert all(torch.equal(same[n], full[n]) for n in full)
    assert all(int(torch.count_nonzero(full[n])) > 0 for n in full)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(37, 64), (13001, 64), (300, 512), (3500, 600), (9, 4096), (3, 16384), (5, 1000), (3500, 333)])
def test_every_operand_that_an_output_may_replace(kind, n, d):
    """out in place of x or the residual, sum_out in place of either, dx in place of x, dout or dsum: the
    bits of the call with outputs of its own."""
    dt = DT[kind]
    g = torch.Generator().manual_seed(n + d)
    x, r, dy, dh = (rows(g, n, d, dt).to(DEV) for _ in range(4))
    w, b = (torch.randn(d, generator=g).to(DEV) for _ in range(2))
    f = rn().rn_layernorm
    out, total = f(x, w, b, residual=r)
    for o, s in (("x", None), ("r", None), ("x", "r"), ("r", "x"), (None, "x"), (None, "r")):
        t = {"x": x.clone(), "r": r.clone()}
        a, c = f(t["x"], w, b, residual=t["r"], out=t.get(o), sum_out=t.get(s))
        assert torch.equal(a, out) and torch.equal(c, total), (o, s)
        assert (o is None or a is t[o]) and (s is None or c is t[s])
        for name, kept in (("x", x), ("r", r)):
            assert name in (o, s) or torch.equal(t[name], kept)
    want = rn().rn_layernorm_backward(dy, x, w, dsum=dh)
    for name in ("x", "dy", "dh"):
        t = {"x": x.clone(), "dy": dy.clone(), "dh": dh.clone()}
        got = rn().rn_layernorm_backward(t["dy"], t["x"], w, dsum=t["dh"], dx=t[name])
        assert all(torch.equal(got[i], want[i]) for i in want), name
        assert all(i == name or torch.equal(t[i], kept) for i, kept in (("x", x), ("dy", dy), ("dh", dh)))


@pytest.mark.parametrize("kind,n,d", [("bf16", 16411, 2568), ("f32", 30001, 96 * 9), ("bf16", 700001, 96), ("bf16", 25001, 2001),
                                      ("f32", 9001, 4999), ("bf16", 300001, 200)])
def test_calls_larger_than_the_caches(kind, n, d):
    """Rows of whole and of broken pieces and lines in calls of more than 256 MB: each row comes out as
    in a call of a few rows. The weights' gradients against float64: sums of at most n / 768 + 1 rows one
    after another, then 24 + 32 of blocks, of products that hold 48 roundings of the normalised value (of
    its own size and of the mean's, at most that of one)."""
    dt = DT[kind]
    g = torch.Generator(DEV).manual_seed(n)
    x, r, dy = (torch.randn(n, d, generator=g, device=DEV).to(dt) for _ in range(3))
    w, b = (torch.randn(d, generator=g, device=DEV) for _ in range(2))
    out, total = rn().rn_layernorm(x, w, b, residual=r)
    got = rn().rn_layernorm_backward(dy, x, w, dsum=r)
    for at in (0, n // 3, n - 40):
        cut = slice(at, at + 40)
        a, c = rn().rn_layernorm(x[cut].clone(), w, b, residual=r[cut].clone())
        assert torch.equal(out[cut], a) and torch.equal(total[cut], c)
        dx = rn().rn_layernorm_backward(dy[cut].clone(), x[cut].clone(), w, dsum=r[cut].clone(), want_dweight=False, want_dbias=False)["dx"]
        assert torch.equal(got["dx"][cut], dx)
    del out, total, r
    xd = x.double()
    xd -= xd.mean(-1, keepdim=True)
    xd /= (xd.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    c = (n / 768 + 1 + 24 + 32 + 48) * U
    dyd = dy.double()
    assert ((got["dbias"] - dyd.sum(0)).abs() <= c * dyd.abs().sum(0)).all()
    assert ((got["dweight"] - (dyd * xd).sum(0)).abs() <= c * (dyd.abs() * (xd.abs() + 1)).sum(0)).all()
