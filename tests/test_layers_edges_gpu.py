"""The head's operators and the optimizer where they can go wrong beside the ordinary sizes: replaced
storage, the ends of the formats' ranges, sides of a limit, calls from threads and other streams.
Tolerances as in ``test_layers_gpu``."""
import math
import threading

import pytest

torch = pytest.importorskip("torch")
from test_layers_gpu import BF, E4, F32, F64, U16, U32, L, check, f32, rand, unpack  # noqa: F401,E402

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
