"""The head's operators and the optimizer where they can go wrong beside the ordinary sizes: replaced
storage, the ends of the formats' ranges, sides of a limit, calls from threads and other streams.
Tolerances as in ``test_layers_gpu``."""
import math
import threading

import pytest

torch = pytest.importorskip("torch")
from test_layers_gpu import (BF, E4, F32, F64, FAST, U16, U32, L, act64, adam64, check, f32, inside, norm_bwd64,  # noqa: F401,E402
                             rand, unpack)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------------- AdamW

def raw(t):
    return t.view(torch.uint8) if t.dtype == E4 else t


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_follows_tensors_whose_storage_is_replaced(L, bits):
    """The step writes where its tensors are now, and not where they were."""
    p, g = [rand(1, 1000), rand(2, 70000)], [rand(3, 1000), rand(4, 70000)]
    copies = [t.bfloat16() for t in p]
    opt = L.AdamW(p, *L.AdamW.new_states(p, bits), copies=copies)
    opt.step(g, lr=1e-2)
    twin_p = [t.clone() for t in p]
    lists = [opt.m, opt.v] + ([opt.m_scale, opt.v_scale] if bits == 8 else [])
    twin_s = [[raw(t).clone().view(t.dtype) for t in ts] for ts in lists]
    twin = L.AdamW(twin_p, *twin_s, copies=[t.clone() for t in copies], step=1)
    everything = [t for ts in [p, copies] + lists for t in ts]
    old = [raw(t.data) for t in everything]
    before = [t.clone() for t in old]
    for t in everything:
        t.data = raw(t.data).clone().view(t.dtype)
    opt.step(g, lr=1e-2)
    twin.step(g, lr=1e-2)
    now = [t for ts in [twin.params, twin.copies] + twin_s for t in ts]
    assert all(torch.equal(raw(a), raw(b)) for a, b in zip(everything, now))
    assert all(torch.equal(a, b) for a, b in zip(old, before))
    assert not torch.equal(p[0], before[0])


def test_adamw_follows_replaced_entries_of_its_lists(L):
    p, g = [rand(1, 500)], [rand(2, 500)]
    opt = L.AdamW(p, *L.AdamW.new_states(p))
    opt.step(g, lr=1e-2)
    m, v, new = opt.m[0].clone(), opt.v[0].clone(), rand(3, 500)
    opt.params[0], opt.m[0], opt.v[0] = new.clone(), m.clone(), v.clone()  # a loaded checkpoint
    opt.step(g, lr=1e-2)
    twin = L.AdamW([new], [m], [v], step=1)
    twin.step(g, lr=1e-2)
    assert torch.equal(opt.params[0], new) and torch.equal(opt.m[0], m) and torch.equal(opt.v[0], v)


def test_adamw_takes_any_iterable(L):
    want, g = [rand(1, 500), rand(2, 300)], [rand(3, 500), rand(4, 300)]
    params = [t.clone() for t in want]
    opt = L.AdamW(want, *L.AdamW.new_states(want, 8), copies=[t.bfloat16() for t in want])
    other = L.AdamW((t for t in params), *(iter(ts) for ts in L.AdamW.new_states(params, 8)),
                    copies=(t.bfloat16() for t in params))
    for _ in range(2):
        opt.step(g, lr=1e-2)
        other.step((t for t in g), lr=1e-2)
    assert all(torch.equal(a, b) for a, b in zip(want, params))


def test_adamw_refuses_tensors_that_no_longer_fit(L):
    p, g = [rand(1, 500)], [rand(2, 500)]
    opt = L.AdamW(p, *L.AdamW.new_states(p))
    p[0].data = rand(3, 400)
    with pytest.raises(ValueError, match="400 elements"):
        opt.step(g, lr=1e-2)
    p[0].data = rand(3, 1000)[::2]
    with pytest.raises(ValueError, match="contiguous"):
        opt.step(g, lr=1e-2)
    p[0].data = rand(3, 500)
    opt.m[0] = opt.m[0].bfloat16()
    with pytest.raises(TypeError, match=r"m\[0\]"):
        opt.step(g, lr=1e-2)
    opt.m[0] = torch.zeros(500)
    with pytest.raises(TypeError, match=r"m\[0\]"):
        opt.step(g, lr=1e-2)
    opt.params.append(rand(4, 3))
    with pytest.raises(ValueError, match="hold 2 tensors"):
        opt.step(g, lr=1e-2)
    assert opt.t == 0


def test_adamw_refuses_buffers_shared_by_two_tensors(L):
    """Two warps of a launch would read and write the same elements.  Gradients may be shared."""
    from contrastive_embedding_loss_gb300.binding import UfError

    p, q, g = rand(1, 500), rand(2, 500), rand(3, 500)

    def step(params, grads, m=None, v=None):
        new_m, new_v = L.AdamW.new_states(params)
        L.AdamW(params, m or new_m, v or new_v).step(grads, lr=1e-2)

    for bad in ([p, p], [p, q, p], [p, p[100:200]]):
        start = p.clone()
        with pytest.raises(UfError, match="invalid-argument"):
            step(bad, [g[:t.numel()] for t in bad])
        assert torch.equal(p, start)
    m = [rand(4, 500)] * 2
    with pytest.raises(UfError, match="invalid-argument"):
        step([p, q], [g, g], m=m)
    with pytest.raises(UfError, match="invalid-argument"):
        step([p, q], [g, p])
    want_p, want_q = p.clone(), q.clone()
    step([want_p], [g])
    step([want_q], [g])
    flat = torch.cat([q, p])  # neighbours in one buffer, in falling order, with one gradient
    step([flat[500:], flat[:500]], [g, g])
    assert torch.equal(flat[500:], want_p) and torch.equal(flat[:500], want_q)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt", [F32, BF])
def test_adamw_bf16_parameters_keep_a_nan(L, bits, gt):
    """Rounding at random adds 16 bits below bf16's own: a NaN stays one."""
    for bad in (float("nan"), float("inf")):
        p, g = [rand(1, 1000, dtype=BF)], rand(2, 1000, dtype=gt)
        g[300] = bad
        L.AdamW(p, *L.AdamW.new_states(p, bits)).step([g], lr=1e-3)
        assert p[0][300].isnan() and int(p[0].isfinite().sum()) == 999


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt", [F32, BF])
@pytest.mark.parametrize("at", [300, 900])
def test_adamw_takes_no_step_where_the_second_moment_overflows(L, bits, pt, at):
    """g = 1e21: v = 0.001 g^2 is infinite in fp32, sqrt(v) too, and m / sqrt(v) is 0."""
    p = [rand(1, 1000, dtype=pt)]
    start = p[0].clone()
    g = rand(2, 1000, scale=1e-3)
    g[at] = 1e21
    opt = L.AdamW(p, *L.AdamW.new_states(p, bits), weight_decay=0.0)
    for _ in range(3):
        opt.step([g], lr=1e-3)
        assert p[0].isfinite().all() and p[0][at] == start[at]
    if bits == 32:
        assert float(opt.v[0][at]) == float("inf") and opt.m[0].isfinite().all()
    else:
        assert opt.m_scale[0].isfinite().all() and opt.v_scale[0].isfinite().sum() == 3
        assert bool((opt.v[0].view(torch.uint8)[at // 256 * 256:][:256] == 126).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-12])
def test_adamw_divides_by_the_root_of_a_subnormal_second_moment(L, bits, eps):
    """g = 3e-19: v = 9e-41 is a multiple of 2^-149.  The first step is lr m / (|g| + eps), m = g."""
    p, g = [torch.zeros(1000, device="cuda")], torch.full((1000,), 3e-19, device="cuda")
    g[::2] *= -1
    opt = L.AdamW(p, *L.AdamW.new_states(p, bits), eps=eps, weight_decay=0.0)
    opt.step([g], lr=1e-2)
    v = 0.001 * float(g[1]) ** 2
    want = -f32(1e-2) * g.to(F64) / (g.to(F64).abs() + f32(eps))
    # the root halves v's relative error: three roundings of at most 2^-150 each
    check("p", p[0], want, want.abs() * (1.5 * 2.0 ** -149 / v + 40 * U32))
    r = opt.v[0].to(F64) * (opt.v_scale[0].to(F64).repeat_interleave(256)[:1000] if bits == 8 else 1)
    want = v ** (0.5 if bits == 8 else 1)
    if eps == 0:
        check("v", r, torch.full_like(r, want), want * (3 * 2.0 ** -150 / v + 16 * U32))


def test_adamw_8bit_momentum_dies_out(L):
    """Without gradients the momentum halves at every step (beta1 = 0.5).  A block whose largest is
    below 2^-116 counts as 0."""
    p, g = [rand(1, 512)], rand(2, 512, scale=1e-3)
    g[256:] = 0
    g[:256:3] = 0
    opt = L.AdamW(p, *L.AdamW.new_states(p, 8), betas=(0.5, 0.999))
    opt.step([g], lr=1e-3)
    zero = torch.zeros_like(g)
    for _ in range(140):
        before = unpack(opt.m[0], opt.m_scale[0])
        opt.step([zero], lr=1e-3)
        m, unit = unpack(opt.m[0], opt.m_scale[0]), opt.m_scale[0].to(F64).repeat_interleave(256)
        # less than one code away, or 0
        check("m", m, before / 2, torch.maximum((before / 2).abs() * 2.0 ** -3, unit * 2.0 ** -9) * 1.0001 + 2.0 ** -116)
        assert not m[before == 0].any()
    assert not opt.m[0].to(F32).any() and not opt.m_scale[0].any()


def test_adamw_counts_its_writes_for_autograd(L):
    """A backward that saved a parameter raises after a step, as with any write in place; an inference
    tensor has no count."""
    p, g = [rand(1, 100).requires_grad_()], [rand(2, 100)]
    opt = L.AdamW(p, *L.AdamW.new_states(p, 8), copies=[p[0].detach().bfloat16()])
    written = [p[0], opt.m[0], opt.v[0], opt.m_scale[0], opt.v_scale[0], opt.copies[0]]
    versions = [t._version for t in written]
    loss = (p[0] * p[0]).sum()
    opt.step(g, lr=1e-2)
    assert all(t._version > v for t, v in zip(written, versions)) and g[0]._version == 0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        p = [rand(1, 100)]
        start = p[0].clone()
        L.AdamW(p, *L.AdamW.new_states(p)).step(g, lr=1e-2)
        assert not torch.equal(p[0], start)


@pytest.mark.parametrize("gt", [F32, BF])
@pytest.mark.parametrize("n,off", [(1000, 0), (1000, 3), (66000, 0)])
def test_adamw_8bit_states_of_bf16_parameters(L, n, off, gt):
    """Parameters and codes are neighbours of the values that they stand for."""
    p, g = rand(1, n + off, dtype=BF)[off:], rand(2, n, scale=1e-2, dtype=gt)
    blocks = -(-n // 256)
    q = [(rand(3 + i, n + off).abs() * 100).clamp(0, 448).to(E4)[off:] for i in range(2)]
    s = [rand(5 + i, blocks).abs() * 1e-4 for i in range(2)]
    m0, r0 = unpack(q[0], s[0]), unpack(q[1], s[1])
    b1, b2, lr, t = 0.9, 0.999, f32(1e-3), 10
    wp, wm, wv = adam64(p, g, m0, r0 * r0, t, lr, b1, b2, f32(1e-8), f32(0.01))
    L.AdamW([p], [q[0]], [q[1]], [s[0]], [s[1]], step=t - 1).step([g], lr=1e-3, seed=77)
    step = lr * (wm.abs() + g.to(F64).abs()) / (1 - b1 ** t) / ((wv / (1 - b2 ** t)).sqrt() + 1e-8)
    # less than one unit away: 2^-7 of the value (16 random bits: a unit's last 2^-16 never rounds up)
    check("p", p, wp, wp.abs() * 2.0 ** -7 * 1.0001 + step * 32 * U32 + 1e-30)
    for name, want, code, scale in (("m", wm, q[0], s[0]), ("v", wv.sqrt(), q[1], s[1])):
        top = torch.nn.functional.pad(want.abs(), (0, blocks * 256 - n)).reshape(blocks, 256).amax(1)
        check(name + " scale", scale, top / 448, top / 448 * 16 * U32 + 1e-40)
        unit = scale.to(F64).repeat_interleave(256)[:n]
        check(name, unpack(code, scale), want, torch.maximum(want.abs() * 2.0 ** -3, unit * 2.0 ** -9) * 1.0001)


def test_adamw_bf16_parameters_and_gradients_in_fp32_states(L):
    p, g = rand(1, 4099, dtype=BF), rand(2, 4099, scale=1e-2, dtype=BF)
    m, v = rand(3, 4099, scale=1e-3), rand(4, 4099, scale=1e-2).square()
    wp, wm, wv = adam64(p, g, m, v, 5, f32(1e-3), eps=f32(1e-8), wd=f32(0.01))
    L.AdamW([p], [m], [v], step=4).step([g], lr=1e-3)
    check("m", m, wm, (wm.abs() + g.to(F64).abs()) * 4 * U32 + 1e-30)
    check("v", v, wv, wv * 6 * U32 + 1e-38)
    slack = 1e-3 * (g.to(F64).abs() + wm.abs()) / (1 - 0.9 ** 5) / ((wv / (1 - 0.999 ** 5)).sqrt() + 1e-8)
    check("p", p, wp, wp.abs() * 2.0 ** -7 * 1.0001 + slack * 32 * U32 + 1e-30)


# ------------------------------------------------------------------------------- RMS norm

def test_rmsnorm_backward_from_two_threads(L):
    """Calls with and without d_stream need rings of different sizes of one kernel; calls from two
    threads may interleave at any point.  (ctypes lets go of the interpreter's lock.)"""
    rows, width, lib = 4, 8192, L._load()
    refused = []

    def calls(carry, seed):
        s, dy, w = rand(seed, rows, width), rand(seed + 1, rows, width), rand(seed + 2, width)
        rstd, dx = torch.ones(rows, device="cuda"), torch.empty(rows, width, device="cuda")
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        bad = 0
        for _ in range(3000):
            bad += 0 != lib.uf_rmsnorm_bwd(dy.data_ptr(), width, 1, s.data_ptr(), width, 1, w.data_ptr(), 1, rstd.data_ptr(),
                                           s.data_ptr() if carry else None, width, rows, width, dx.data_ptr(), width, None,
                                           None, 0, stream.cuda_stream)
        stream.synchronize()
        refused.append(bad)

    threads = [threading.Thread(target=calls, args=(carry, 10 * carry)) for carry in (False, True)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == [0, 0]


@pytest.mark.parametrize("width", [77, 520, 5000])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_rmsnorm_e4m3_rows_of_tiny_values(L, width, dtype):
    """y is up to 1000 times s (rho = eps^-1/2): rows whose s are below 448 / 2^128 have a larger y."""
    x = rand(1, 6, width) * torch.tensor([1e-36, 1e-37, 2e-38, 1.0, 1e-30, 0.0], device="cuda")[:, None]
    x = x.to(dtype)
    x[:, 1::3] = 0
    w = 1 + rand(2, width, scale=0.1)
    got = L.rmsnorm_fwd(x, w, eps=1e-6, out="e4m3")
    y = x.to(F64) * (x.to(F64).square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.to(F64)
    top, rel = y.abs().amax(1), (width / 2 + 24) * U32
    check("scale", got["scale"], top / 448, top / 448 * (rel + 4 * U32))
    scale = got["scale"].to(F64)[:, None]
    check("y", got["y"].to(F64) * scale, y, torch.maximum(y.abs() * 2.0 ** -4, scale * 2.0 ** -10) * 1.001 + y.abs() * rel)


def test_rmsnorm_e4m3_rows_below_the_range_count_as_zeros(L):
    x = rand(1, 3, 200)
    x[1] *= 1e-41
    x[1, ::2] = 0
    got = L.rmsnorm_fwd(x, torch.ones(200, device="cuda"), eps=1e-6, out="e4m3")
    assert float(got["scale"][1]) == 0 and not got["y"][1].to(F32).any()
    assert bool((got["scale"][::2] > 0).all())


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 1e30])
def test_rmsnorm_e4m3_marks_a_non_finite_row(L, bad):
    """An infinity or a NaN makes its row's products NaN, as the formula does; where only the mean of
    squares overflows, rho is 0 and so is the row."""
    x = rand(1, 3, 520)
    clean = L.rmsnorm_fwd(x, torch.ones(520, device="cuda"), out="e4m3")
    x[1, 100] = bad
    got = L.rmsnorm_fwd(x, torch.ones(520, device="cuda"), out="e4m3")
    y = got["y"].to(F32) * got["scale"][:, None]
    assert torch.equal(got["y"].view(torch.uint8)[::2], clean["y"].view(torch.uint8)[::2])
    assert y[1].isnan().all() if bad != 1e30 else not y[1].any()


def norm_bwd_check(L, dy, s, w, ds):
    rows, width = s.shape
    rho = (s.to(F64).square().mean(1) + 1e-6).rsqrt().to(F32)
    got = L.rmsnorm_bwd(dy, s, w, rho, d_stream=ds)
    dx, size, dw, dw_size = norm_bwd64(dy.to(F64), s.to(F64), w.to(F64), rho.to(F64), None if ds is None else ds.to(F64))
    check("dx", got["dx"], dx, size * (width + 16) * U32 + (dx.abs() * U16 if s.dtype == BF else 0) + 1e-30)
    check("dweight", got["dweight"], dw, dw_size * (rows + 16) * U32 + 1e-30)


# For each number of threads a row: odd widths, whose rows start at every alignment, and rows enough
# that a block takes several, 8 or a multiple apart.
MANY_ROWS = [(3001, 77), (3003, 515), (3001, 1023), (5003, 1031), (1300, 2051), (1300, 4099), (700, 8191), (700, 16383)]


@pytest.mark.parametrize("rows,width", MANY_ROWS)
@pytest.mark.parametrize("dyt,st,carry", [(BF, BF, True), (F32, F32, False), (BF, F32, True), (F32, BF, False)])
def test_rmsnorm_bwd_of_many_rows_of_odd_width(L, rows, width, dyt, st, carry):
    dy, s = rand(2, rows, width, dtype=dyt), rand(1, rows, width, dtype=st)
    norm_bwd_check(L, dy, s, 1 + rand(3, width, scale=0.1), rand(4, rows, width, dtype=st) if carry else None)


@pytest.mark.parametrize("rows,width", [(3001, 500), (700, 4100)])
@pytest.mark.parametrize("st", [BF, F32])
def test_rmsnorm_bwd_of_rows_with_an_odd_pitch(L, rows, width, st):
    """All arrays in step with one another, in rows of width + 5 elements: so is the returned dx's
    misalignment to theirs, and the accesses are single elements unless dx has the same pitch."""
    dy, s, ds = (rand(i, rows, width + 5, dtype=t)[:, :width] for i, t in ((1, BF), (2, st), (3, st)))
    norm_bwd_check(L, dy, s, 1 + rand(4, width, scale=0.1), ds)
    # through the C ABI into a dx of that pitch: vectors from a row's first boundary on
    lib, pitch = L._load(), width + 5
    rho = (s.to(F64).square().mean(1) + 1e-6).rsqrt().to(F32)
    w, dw = 1 + rand(4, width, scale=0.1), torch.empty(width, device="cuda")
    dx = torch.full((rows, pitch), 7.0, device="cuda").to(st)
    ws = torch.empty(lib.uf_rmsnorm_bwd_workspace(rows, width), dtype=torch.uint8, device="cuda")
    kind = 0 if st == BF else 1
    assert 0 == lib.uf_rmsnorm_bwd(dy.data_ptr(), pitch, 0, s.data_ptr(), pitch, kind, w.data_ptr(), 1, rho.data_ptr(),
                                   ds.data_ptr(), pitch, rows, width, dx.data_ptr(), pitch, dw.data_ptr(), ws.data_ptr(),
                                   ws.numel(), torch.cuda.current_stream().cuda_stream)
    want, size, dw64, dw_size = norm_bwd64(dy.to(F64), s.to(F64), w.to(F64), rho.to(F64), ds.to(F64))
    check("dx", dx[:, :width], want, size * (width + 16) * U32 + (want.abs() * U16 if st == BF else 0) + 1e-30)
    check("dweight", dw, dw64, dw_size * (rows + 16) * U32 + 1e-30)
    assert bool((dx[:, width:] == 7.0).all())


@pytest.mark.parametrize("rows,width", [(1300, 600), (700, 1500), (700, 5000), (400, 9000)])
@pytest.mark.parametrize("st", [BF, F32])
def test_rmsnorm_out_of_step(L, rows, width, st):
    """Arrays whose 16-byte boundaries lie at different elements: single elements, 32 to 512 threads a row."""
    x, r = inside(rand(1, rows, width, dtype=BF), pad_cols=3), rand(2, rows, width, scale=2.0, dtype=st)
    w = 1 + rand(3, width, scale=0.1, dtype=BF)
    for out in ("bf16", "e4m3"):
        got = L.rmsnorm_fwd(x, w, residual=r, out=out)
        s = x.to(F64) + r.to(F64)
        y = s * (s.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.to(F64)
        rel = (width / 2 + 24) * U32
        check("stream", got["stream"], s, s.abs() * (U16 * 1.01 if st == BF else 2 * U32) + 1e-30)
        if out == "bf16":
            check("y", got["y"], y, y.abs() * (U16 + 2 * rel) + 1e-30)
        else:
            scale = got["scale"].to(F64)[:, None]
            check("y", got["y"].to(F64) * scale, y, torch.maximum(y.abs() * 2.0 ** -4, scale * 2.0 ** -10) * 1.001 + y.abs() * rel)
    norm_bwd_check(L, inside(rand(4, rows, width, dtype=BF), pad_cols=3), r, w, rand(5, rows, width, dtype=st))


@pytest.mark.parametrize("width", [1000, 1001])
def test_rmsnorm_bwd_of_a_bf16_weight(L, width):
    norm_bwd_check(L, rand(1, 300, width, dtype=BF), rand(2, 300, width), 1 + rand(3, width, scale=0.1, dtype=BF), None)


# -------------------------------------------------------------------------------- products

@pytest.mark.parametrize("rows", [5, 300, 3000])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_bwd_of_what_is_asked(L, rows, act):
    inner, outer = 264, 520
    x, w, dy = rand(1, rows, inner, dtype=BF), rand(2, outer, inner, dtype=BF), rand(3, rows, outer, dtype=BF)
    pre = rand(4, rows, outer, dtype=BF) if act != "none" else None
    da = 1.0 if pre is None else act64(pre.to(F64), act)[1]
    dz = dy.to(F64) * da
    off = torch.zeros_like(dz) if pre is None else dy.to(F64).abs() * 4 * FAST
    rounded = off + (0 if pre is None else dz.abs() * U16)
    X, W = x.to(F64), w.to(F64)
    want = {"dx": dz @ W, "dW": dz.t() @ X, "dbias": dz.sum(0)}
    bound = {"dx": rounded @ W.abs() * 1.01 + dz.abs() @ W.abs() * (outer + 8) * 2 * U32 + want["dx"].abs() * U16 * 1.01 + 1e-30,
             "dW": rounded.t() @ X.abs() * 1.01 + dz.abs().t() @ X.abs() * (rows + 8) * 2 * U32 + want["dW"].abs() * U16 * 1.01 + 1e-30,
             "dbias": off.sum(0) + dz.abs().sum(0) * (rows + 8) * U32 + 1e-30}
    for need in (("dx",), ("dW",), ("dbias",), ("dx", "dbias"), ("dW", "dbias"), ("dx", "dW"), ()):
        got = L.linear_bwd(dy, x, w, pre=pre, act=act, need=need)
        assert set(got) == set(need)
        for k in need:
            check(f"{k} of {need}", got[k], want[k], bound[k])
    with pytest.raises(ValueError, match="need names"):
        L.linear_bwd(dy, x, w, need=("dy",))


@pytest.mark.parametrize("rows", [5, 300, 3000])
def test_gated_bwd_of_what_is_asked(L, rows):
    inner, outer = 264, 136
    x, w, dh = rand(1, rows, inner, dtype=BF), rand(2, 2 * outer, inner, dtype=BF), rand(3, rows, outer, dtype=BF)
    pre = rand(4, rows, 2 * outer, dtype=BF)
    g, u = pre.to(F64).split(outer, 1)
    a, da = act64(g, "silu")
    d = torch.cat([dh.to(F64) * u * da, dh.to(F64) * a], 1)
    err = torch.cat([(dh.to(F64) * u).abs() * 4 * FAST, (dh.to(F64) * g).abs() * FAST], 1) + d.abs() * U16 * 1.01
    X, W = x.to(F64), w.to(F64)
    want = {"dx": d @ W, "dW": d.t() @ X}
    bound = {"dx": err @ W.abs() + d.abs() @ W.abs() * (2 * outer + 8) * 2 * U32 + want["dx"].abs() * U16 * 1.01 + 1e-30,
             "dW": err.t() @ X.abs() + d.abs().t() @ X.abs() * (rows + 8) * 2 * U32 + want["dW"].abs() * U16 * 1.01 + 1e-30}
    for need in (("dx",), ("dW",), ("dx", "dW"), ()):
        got = L.gated_bwd(dh, x, w, pre, need=need)
        assert set(got) == set(need)
        for k in need:
            check(f"{k} of {need}", got[k], want[k], bound[k])


def test_the_callers_workspace_and_status(L):
    from contrastive_embedding_loss_gb300.binding import UfError

    lib = L._load()
    x, w, dy = rand(1, 64, 8192, dtype=BF), rand(2, 256, 8192, dtype=BF), rand(3, 64, 256, dtype=BF)
    pre, rstd, n = rand(4, 64, 256, dtype=BF), torch.ones(64, device="cuda"), torch.ones(256, device="cuda")
    calls = {  # (call, its scratch, whether it takes a status word)
        "rmsnorm_bwd": (lambda **k: L.rmsnorm_bwd(dy, pre, n, rstd, **k), lib.uf_rmsnorm_bwd_workspace(64, 256), False),
        "linear_fwd": (lambda **k: L.linear_fwd(x, w, **k), lib.uf_linear_fwd_workspace(64, 8192, 256, 0), True),
        "linear_bwd": (lambda **k: L.linear_bwd(dy, x, w, pre=pre, act="silu", **k), lib.uf_linear_bwd_workspace(64, 8192, 256), True),
        "gated_fwd": (lambda **k: L.gated_fwd(x, w, **k), lib.uf_gated_fwd_workspace(64, 8192, 128), True),
        "gated_bwd": (lambda **k: L.gated_bwd(dy[:, :128], x, w, pre, **k), lib.uf_gated_bwd_workspace(64, 8192, 128), True),
    }
    for name, (call, need, takes_status) in calls.items():
        assert need > 0, name
        want = call()
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = call(workspace=ws[:need], **({"device_status": status} if takes_status else {}))
        assert all(torch.equal(got[k], want[k]) for k in want), name
        assert int(status) == 0 and bool((ws[need:] == 255).all()), name
        with pytest.raises(UfError, match="workspace-too-small"):
            call(workspace=ws[:need - 1])
        with pytest.raises(UfError, match="invalid-argument"):
            call(workspace=ws[16:])  # not on 256 bytes
        for bad in (ws.float(), ws[::2], ws.cpu(), need):
            with pytest.raises(TypeError, match="workspace"):
                call(workspace=bad)
        if takes_status:
            for bad in (status.float(), status.cpu(), status[:0], 0):
                with pytest.raises(TypeError, match="device_status"):
                    call(device_status=bad)


# ---------------------------------------------------------------------------- activations

@pytest.mark.parametrize("rows", [4, 40])
def test_gelu_in_its_negative_tail(L, rows):
    """gelu and its derivative for z from -3 down to -12, relative to their values: a rounding to bf16, and
    2^-12 for the fp32 value (1.4e-4 of the fit, 1e-5 of the exponential's argument)."""
    z = -torch.linspace(3, 12, rows, device="cuda").to(BF)
    x, w = torch.zeros(rows, 64, dtype=BF, device="cuda"), torch.zeros(64, 64, dtype=BF, device="cuda")
    x[:, 5], w[:, 5] = z, 1  # every output's argument is z itself
    z = z.to(F64)
    cdf = torch.special.erfc(-z / math.sqrt(2)) / 2
    want = (z * cdf)[:, None].expand(rows, 64)
    check("gelu", L.linear_fwd(x, w, act="gelu")["y"], want, want.abs() * (U16 * 1.01 + 2.0 ** -12))
    want = want * z[:, None]
    check("gated", L.gated_fwd(x, torch.cat([w, w]), act="gelu")["h"], want, want.abs() * (U16 * 1.01 + 2.0 ** -12))
    da = cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    dy, one = torch.ones(1, 64, device="cuda"), x[:1]
    for r in range(rows):
        pre = z[r].to(BF).expand(1, 64).contiguous()
        got = L.linear_bwd(dy, one, w, pre=pre, act="gelu", need=("dbias",))["dbias"]
        check("gelu'", got, da[r].expand(64), da[r].abs() * 2.0 ** -12)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_of_large_arguments(L, act):
    """Far from 0 every activation is 0 or z, with a derivative of 0 or 1, up to the largest bf16."""
    z = torch.tensor([[40.0, 1e4, 1e13, 3e19, 1e30, 3e38], [-200.0, -1e4, -1e13, -3e19, -1e30, -3e38]], device="cuda").to(BF)
    z = torch.cat([z, z[:, :2]], 1)
    x, w = torch.zeros(2, 64, dtype=BF, device="cuda"), torch.zeros(8, 64, dtype=BF, device="cuda")
    x[:, 3], w[:, 3] = z[:, 0], 1
    for c in range(8):
        x[:, 3] = z[:, c]
        y = L.linear_fwd(x, w, act=act)["y"]
        assert bool((y[0] == z[0, c]).all()) and bool((y[1] == 0).all())
    for r, want in ((0, 1.0), (1, 0.0)):
        dy = torch.ones(1, 8, device="cuda")
        got = L.linear_bwd(dy, x[:1], w, pre=z[r:r + 1].contiguous(), act=act, need=("dbias", "dx"))
        assert bool((got["dbias"] == want).all()) and bool((got["dx"][:, 3] == 8 * want).all())
        got = L.gated_bwd(dy.to(BF), x[:1], torch.cat([w, w]), torch.cat([z[r:r + 1], torch.ones_like(z[:1])], 1), act=act,
                          need=("dx",))
        assert got["dx"].isfinite().all()

# ---------------------------------------------------------------------------- other streams

def test_inputs_of_a_call_on_another_stream_may_be_freed(L):
    """Calls that wait behind a long kernel on their stream; their inputs are freed and as much memory
    is allocated and overwritten on the current stream meanwhile."""
    args = {"x": rand(1, 300, 512, dtype=BF), "w": rand(2, 256, 512, scale=0.05, dtype=BF), "n": rand(3, 512),
            "r": rand(4, 300, 512), "dy": rand(5, 300, 256, dtype=BF), "pre": rand(6, 300, 256, dtype=BF),
            "dh": rand(7, 300, 128, dtype=BF), "rstd": rand(8, 300).abs(), "p": rand(9, 1 << 16), "g": rand(10, 1 << 16),
            "lr": torch.full((1,), 0.5, device="cuda")}
    passes = {
        "rmsnorm_fwd": (lambda a, s: L.rmsnorm_fwd(a["x"], a["n"], residual=a["r"], stream=s), "x n r"),
        "rmsnorm_bwd": (lambda a, s: L.rmsnorm_bwd(a["x"], a["r"], a["n"], a["rstd"], d_stream=a["r"], stream=s), "x r n rstd"),
        "linear_fwd": (lambda a, s: L.linear_fwd(a["x"], a["w"], bias=a["n"][:256], residual=a["dy"], stream=s), "x w n dy"),
        "linear_bwd": (lambda a, s: L.linear_bwd(a["dy"], a["x"], a["w"], pre=a["pre"], act="gelu", stream=s), "dy x w pre"),
        "gated_fwd": (lambda a, s: L.gated_fwd(a["x"], a["w"], stream=s), "x w"),
        "gated_bwd": (lambda a, s: L.gated_bwd(a["dh"], a["x"], a["w"], a["pre"], stream=s), "dh x w pre"),
    }

    def adamw(a, s):
        opt = L.AdamW([a["p"]], *L.AdamW.new_states([a["p"]]))
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())  # (the states)
        opt.step((a["g"],), lr=a["lr"], stream=s)
        return {"p": a["p"]}

    passes["adamw"] = (adamw, "g lr")
    side = torch.cuda.Stream()
    for name, (call, names) in passes.items():
        want = call({k: t.clone() for k, t in args.items()}, None)
        a = {k: t.clone() for k, t in args.items()}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(a, side)
        freed = [(a[k].shape, a[k].dtype) for k in names.split()]
        for k in names.split():
            del a[k]
        junk = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for shape, dtype in freed]
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want), name
        del junk


# -------------------------------------------------------------------------------- refusals

def test_widths_past_32_bits_are_refused(L):
    """A width of 2^32 + 8 is not one of 8."""
    wide = (1 << 32) + 8
    rows = torch.empty(0, wide, dtype=BF, device="cuda")
    w = torch.empty(wide, dtype=BF, device="cuda")
    for call in (lambda: L.rmsnorm_fwd(rows, w), lambda: L.rmsnorm_bwd(rows, rows, w, torch.empty(0, device="cuda"))):
        with pytest.raises(ValueError, match="width may be at most"):
            call()
    x = torch.empty(0, 8, dtype=BF, device="cuda")
    del w
    W = torch.empty(wide, 8, dtype=BF, device="cuda")  # 64 GiB, never written
    with pytest.raises(ValueError, match="rows may be at most"):
        L.linear_fwd(x, W)
    with pytest.raises(ValueError, match="rows may be at most"):
        L.gated_fwd(x, W)
    del W
    torch.cuda.empty_cache()
