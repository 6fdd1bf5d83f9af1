"""Token log probabilities, entropies, top alternatives and their gradient:
refusals and the oracle on the CPU, parity on the GPU.

Tolerances, with u = 2^-24 (half a step of fp32).  Forward: d = (z - max) is
rounded a few times (relative 4 u), which moves s = sum e^d by at most
4 u sum |d| e^d <= 4 u s (ln V + 1); ex2.approx adds 2^-22 = 4 u per term; a
thread adds at most V / 256 + 64 terms one after another (u each).  So ln s is
off by at most (4 (ln V + 1) + 4 + V / 256 + 64 + 1) u, and a difference or
product on the way out adds 4 u of its value and of the largest |z| (lse).
t / s is a mean of d under p, with the same relative error per term.
Gradient: log p = z scale - lse carries u (|z| + 2 |lse|) from lse's own
rounding and the fused multiply-add, ex2 its argument's rounding u |log p| and
4 u; then one round to the output type, eps / 2 of the value.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
import rmsnorm_linear_projection_flashnorm_b200 as fnb
from rmsnorm_linear_projection_flashnorm_b200 import torch_api as T

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
A, B, C, D, E = (1 << 30), (1 << 34), (1 << 35), (1 << 36), (1 << 37)


# ------------------------------------------------------------------ CPU: refusals
@pytest.fixture(scope="module", autouse=True)
def _lib():
    fnb.build()
    fnb.lib()


def fwd_(logits=A, type=0, M=4, V=1000, ld=1000, t=B, scale=1.0, k=5, lp=C, H=C + 64, lse=C + 128, ids=D, top=E):
    return fnb.fn_token_logprobs(logits, type, M, V, ld, t, scale, k, lp, H, lse, ids, top, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), fnb.FN_ERR_INVALID_ARG),
    (dict(V=0), fnb.FN_ERR_INVALID_ARG),
    (dict(ld=999), fnb.FN_ERR_INVALID_ARG),
    (dict(type=3), fnb.FN_ERR_INVALID_ARG),
    (dict(scale=0.0), fnb.FN_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fnb.FN_ERR_INVALID_ARG),
    (dict(scale=float("inf")), fnb.FN_ERR_INVALID_ARG),
    (dict(k=-1), fnb.FN_ERR_INVALID_ARG),
    (dict(k=4, V=3, ld=3), fnb.FN_ERR_INVALID_ARG),
    (dict(k=33), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(M=1 << 28), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(V=1 << 31, ld=1 << 31), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(logits=None), fnb.FN_ERR_INVALID_ARG),
    (dict(t=None), fnb.FN_ERR_INVALID_ARG),
    (dict(ids=None), fnb.FN_ERR_INVALID_ARG),
    (dict(top=None), fnb.FN_ERR_INVALID_ARG),
    (dict(k=0), fnb.FN_ERR_INVALID_ARG),                       # top outputs without a top_k
    (dict(k=0, ids=None, top=None, lp=None, H=None, lse=None), fnb.FN_ERR_INVALID_ARG),
    (dict(logits=A + 1), fnb.FN_ERR_ALIGNMENT),
    (dict(type=2, logits=A + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(t=B + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(lse=C + 130), fnb.FN_ERR_ALIGNMENT),
    (dict(lp=A + 4), fnb.FN_ERR_ALIAS),
    (dict(H=C + 8), fnb.FN_ERR_ALIAS),                         # entropy overlaps logprob
    (dict(top=D + 40), fnb.FN_ERR_ALIAS),                      # 4 x 5 ids: 80 bytes
    (dict(ids=B + 12), fnb.FN_ERR_ALIAS),
])
def test_forward_refusals(kw, code):
    assert fwd_(**kw) == code


def bwd_(logits=A, type=0, M=4, V=1000, ld=1000, t=B, lse=C, H=C + 64, gl=C + 128, gh=C + 192, scale=1.0, d=D, ldd=1000):
    return fnb.fn_token_logprobs_backward(logits, type, M, V, ld, t, lse, H, gl, gh, scale, d, ldd, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), fnb.FN_ERR_INVALID_ARG),
    (dict(ldd=999), fnb.FN_ERR_INVALID_ARG),
    (dict(type=-1), fnb.FN_ERR_INVALID_ARG),
    (dict(scale=-1.0), fnb.FN_ERR_INVALID_ARG),
    (dict(lse=None), fnb.FN_ERR_INVALID_ARG),
    (dict(d=None), fnb.FN_ERR_INVALID_ARG),
    (dict(t=None), fnb.FN_ERR_INVALID_ARG),
    (dict(H=None), fnb.FN_ERR_INVALID_ARG),
    (dict(gl=None, gh=None), fnb.FN_ERR_INVALID_ARG),
    (dict(M=(1 << 31) - 1, V=100000, ld=100000, ldd=100000), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(d=D + 1), fnb.FN_ERR_ALIGNMENT),
    (dict(gl=C + 129), fnb.FN_ERR_ALIGNMENT),
    (dict(d=A + 2), fnb.FN_ERR_ALIAS),                         # overlaps the logits, not in place
    (dict(d=A, ldd=1001), fnb.FN_ERR_ALIAS),                   # in place with another row stride
    (dict(d=C - 4000), fnb.FN_ERR_ALIAS),                      # overlaps lse
])
def test_backward_refusals(kw, code):
    assert bwd_(**kw) == code


def test_empty_batch_is_a_noop():
    assert fwd_(M=0, logits=None, t=None) == fnb.FN_OK
    assert bwd_(M=0, logits=None, lse=None, d=None) == fnb.FN_OK


def test_torch_api_refuses_what_the_library_cannot_see():
    x = torch.zeros(2, 8)
    t = torch.zeros(2, dtype=torch.int32)
    for bad in (lambda: T.token_logprobs(x, t),                                # not on a GPU
                lambda: T.token_logprobs(x.double(), t),
                lambda: T.token_logprobs(x[0], t),
                lambda: T.token_logprobs(x, t.long()),
                lambda: T.token_logprobs(x, t[:1]),
                lambda: T.token_logprobs(x.t().contiguous().t(), t),
                lambda: T.token_logprobs_backward(x, t, torch.zeros(3), None, torch.zeros(2)),
                lambda: T.token_logprobs_backward(x, t, torch.zeros(2), None, torch.zeros(2).double()),
                lambda: T.token_logprobs_backward(x, t, torch.zeros(2), None, torch.zeros(2), out=x.half())):
        with pytest.raises(ValueError):
            bad()


# ------------------------------------------------------------------ CPU: the oracle
def test_oracle_against_brute_force_and_differences():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 7))
    x[1, 2] = -np.inf
    t = np.array([3, 0, -1])
    lp, H, lse, ids, top = O.token_logprobs(x, t, 3, 0.5)
    p = np.exp(0.5 * x) / np.exp(0.5 * x).sum(1, keepdims=True)
    assert np.allclose(lp, [math.log(p[0, 3]), math.log(p[1, 0]), 0.0], atol=1e-13)
    assert np.allclose(H, [-sum(v * math.log(v) for v in r if v > 0) for r in p], atol=1e-13)
    assert np.allclose(np.exp(lse), np.exp(0.5 * x).sum(1))
    assert np.array_equal(ids[0], np.argsort(-x[0])[:3]) and np.allclose(np.exp(top[0]), np.sort(p[0])[::-1][:3])
    gl, gh = rng.standard_normal(3), rng.standard_normal(3)
    g = O.token_logprobs_grad(x, t, gl, gh, 0.5)
    f = lambda z: (lambda r: np.sum(gl * r[0]) + np.sum(gh * r[1]))(O.token_logprobs(z, t, 0, 0.5))
    for i in range(3):
        for j in range(7):
            if np.isfinite(x[i, j]):
                e = np.zeros_like(x)
                e[i, j] = 1e-6
                assert abs((f(x + e) - f(x - e)) / 2e-6 - g[i, j]) < 1e-8


def test_oracle_order_of_ties_and_nan():
    x = np.array([[1.0, 2.0, 2.0, 0.0, -0.0, 1.0]])
    assert O.token_logprobs(x, None, 6)[3].tolist() == [[1, 2, 0, 5, 3, 4]]
    x = np.array([[1.0, np.nan, np.inf, np.nan, -np.inf]])
    assert O.token_logprobs(x, None, 5)[3].tolist() == [[1, 3, 2, 0, 4]]


# ------------------------------------------------------------------ GPU: parity
def logits_(M, V, ld, dtype, seed, spread=3.0, masked=0.0, offset=0):
    gen = torch.Generator().manual_seed(seed)
    buf = torch.randn(M * ld + offset, generator=gen) * spread
    if masked:
        buf[torch.rand(buf.shape, generator=gen) < masked] = -math.inf
    buf = buf.to(DT[dtype]).cuda()
    return buf[offset:].view(M, ld)[:, :V]


def targets_(M, V, seed):
    rng = np.random.default_rng(seed)
    t = rng.integers(0, V, M).astype(np.int32)
    if M > 2:
        t[1] = -1
    return t


def check_fwd(x, t, k, scale):
    r = T.token_logprobs(x, torch.from_numpy(t).cuda(), top_k=k, scale=scale)
    torch.cuda.synchronize()
    xc = x.float().cpu()
    lp, H, lse, ids, top = O.token_logprobs(xc, t, k, scale)
    V = x.shape[1]
    ls = (4 * (math.log(V) + 1) + V / 256 + 69) * U
    with np.errstate(all="ignore"):
        big = np.nan_to_num(np.abs(np.where(np.isfinite(xc.numpy()), xc.numpy(), 0.0)).max(1) * scale)
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)

    def close(got, ref, tol):
        got, ref = got.cpu().double().numpy(), np.asarray(ref)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        fin = np.isfinite(ref)
        assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
        tol = np.broadcast_to(tol, ref.shape)
        assert np.all(np.abs(got[fin] - ref[fin]) <= tol[fin]), np.max(np.abs(got[fin] - ref[fin]) - tol[fin])

    fin = lambda a: np.where(np.isfinite(a), np.abs(a), 0.0)
    close(r.logprob, lp, ls + 4 * U * (fin(lp) + 1) + 4 * U * fin(lp))
    close(r.lse, lse, ls + 4 * U * (fin(lse) + big))
    close(r.entropy, H, 2 * ls * (1 + math.log(V)) + 4 * U * (fin(H) + 1))
    close(r.top_logprobs, top, ls + 8 * U * (fin(top) + 1))
    return r


SHAPES = [(1, 1), (1, 2), (3, 5), (2, 31), (5, 257), (4, 1000), (1, 8192), (3, 8193), (2, 16384 + 9), (1, 50021),
          (1, 131072), (40, 32003), (700, 4099)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,V", SHAPES)
def test_forward(M, V, dtype):
    x = logits_(M, V, V + (M > 1) * (V % 3), dtype, seed=M * 1000 + V, offset=V % 5)
    check_fwd(x, targets_(M, V, V), min(V, 20), 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [0, 1, 2, 31, 32])
def test_forward_top_k(k):
    check_fwd(logits_(3, 40000, 40000, "bf16", seed=k), targets_(3, 40000, k), k, 0.7)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.25, 3.0])
@pytest.mark.parametrize("masked", [0.3, 0.999])
def test_forward_masked(masked, scale):
    x = logits_(5, 30011, 30011, "fp32", seed=1, masked=masked)
    x[3] = -math.inf                       # nothing left
    x[4, 1:] = -math.inf                   # one token left
    x[4, 0] = 2.0
    t = targets_(5, 30011, 2)
    t[4] = 0
    check_fwd(x, t, 32, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["up", "down", "flat", "steps", "saw"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_orders(order, dtype):
    """Rows that grow steadily (every tile overflows the survivor buffer), fall,
    are constant (ties everywhere), or tie in long runs."""
    V = 70001
    i = torch.arange(V, dtype=torch.float32)
    row = {"up": i / V * 20 - 10, "down": 10 - i / V * 20, "flat": torch.full((V,), 0.5),
           "steps": torch.floor(i / 5000) - 7, "saw": (i % 64) / 8}[order]
    x = row.to(DT[dtype]).expand(3, V).contiguous().cuda()
    check_fwd(x, targets_(3, V, 0), 32, 1.0)


@pytest.mark.gpu
def test_forward_signed_zeros_infinities_and_nan():
    x = torch.zeros(6, 9000)
    x[0, ::2] = -0.0                       # -0 ties with +0
    x[1, 17] = math.nan
    x[2, 8999] = math.inf
    x[3, 5] = math.nan
    x[3, 8000] = math.inf
    x[4] = torch.finfo(torch.float32).min  # masked by the type's lowest value: uniform
    x[5, 1:] = torch.finfo(torch.float32).min
    t = np.array([1, 2, 3, 4, 5, 0], dtype=np.int32)
    x = x.cuda()
    r = T.token_logprobs(x, torch.from_numpy(t).cuda(), top_k=4)
    torch.cuda.synchronize()
    lp, H, lse, ids, top = O.token_logprobs(x.cpu(), t, 4)
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    for got, ref in ((r.logprob, lp), (r.entropy, H), (r.lse, lse), (r.top_logprobs, top)):
        got = got.cpu().double().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        ok = ~np.isnan(ref)
        assert np.allclose(got[ok], ref[ok], rtol=1e-5, atol=1e-5)


@pytest.mark.gpu
def test_forward_target_out_of_range_and_optional_outputs():
    x = logits_(3, 100, 100, "bf16", seed=3)
    t = torch.tensor([100, 2**31 - 1, -2**31], dtype=torch.int32, device="cuda")
    lp = T.token_logprobs(x, t).logprob.cpu()
    assert torch.isnan(lp[:2]).all() and lp[2] == 0
    r = T.token_logprobs(x)
    assert r.logprob is None and r.top_ids.shape == (3, 0)
    # each output alone
    for i in range(4):
        o = [torch.full((3,), 7.0, device="cuda") if j == i else None for j in range(3)]
        ids = torch.empty((3, 2), dtype=torch.int32, device="cuda") if i == 3 else None
        top = torch.empty((3, 2), device="cuda") if i == 3 else None
        fnb.check(fnb.fn_token_logprobs(x, 0, 3, 100, 100, t, 1.0, 2 if i == 3 else 0, *o, ids, top))
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_rows_behind_the_outputs_stay_and_repeats_are_equal():
    x = logits_(9, 20011, 20011, "bf16", seed=5)
    t = torch.from_numpy(targets_(9, 20011, 1)).cuda()
    f = torch.full((4, 12), 9.0, device="cuda")
    ids = torch.full((12, 8), 9, dtype=torch.int32, device="cuda")
    top = torch.full((12, 8), 9.0, device="cuda")
    runs = []
    for _ in range(3):
        out = T.TokenLogprobs(f[0, :9], f[1, :9], f[2, :9], ids[:9], top[:9])
        T.token_logprobs(x, t, top_k=8, out=out)
        torch.cuda.synchronize()
        runs.append([v.clone() for v in out])
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))
    assert (f[:3, 9:] == 9).all() and (f[3] == 9).all() and (ids[9:] == 9).all() and (top[9:] == 9).all()


def check_bwd(x, t, gl, gh, scale, out=None):
    tg = torch.from_numpy(t).cuda()
    ref = O.token_logprobs_grad(x.float().cpu(), t, gl, gh, scale)
    xc = np.abs(np.where(np.isfinite(x.float().cpu().numpy()), x.float().cpu().numpy(), 0.0)) * scale
    r = T.token_logprobs(x, tg, scale=scale)
    cu = lambda a: None if a is None else torch.from_numpy(a).cuda()
    lse = np.nan_to_num(r.lse.cpu().numpy().astype(np.float64), neginf=0.0)
    Hn = r.entropy.cpu().numpy().astype(np.float64)
    g = T.token_logprobs_backward(x, tg, r.lse, r.entropy, cu(gl), cu(gh), scale=scale, out=out)
    torch.cuda.synchronize()
    got = g.double().cpu().numpy()
    V = x.shape[1]
    ls = (4 * (math.log(V) + 1) + V / 256 + 69) * U            # lse's own error
    eh = 2 * ls * (1 + math.log(V)) + 4 * U * (Hn[:, None] + 1)
    elp = ls + U * (2 * xc + 4 * np.abs(lse)[:, None])         # error of log p
    lp = xc + np.abs(lse)[:, None]
    rel_p = elp + 4 * U + 2 * U * lp
    agl = np.abs(gl)[:, None] if gl is not None else 0.0
    agh = np.abs(gh)[:, None] if gh is not None else 0.0
    p = np.minimum(1.0, np.exp(np.minimum(0.0, np.where(np.isfinite(x.float().cpu().numpy()),
                                                       x.float().cpu().numpy() * scale - lse[:, None], -np.inf))))
    tol = scale * p * (agl * (rel_p + 4 * U) + agh * ((lp + Hn[:, None]) * (rel_p + 4 * U) + elp + eh))
    tol = tol + scale * agl * 4 * U + torch.finfo(x.dtype).eps / 2 * np.abs(ref) * (1 + 2 ** -10)
    tol = tol + {torch.float16: 2.0 ** -25}.get(x.dtype, 0.0)  # fp16 subnormals: half a step
    tol = tol + 2.0 ** -126                                    # ex2 flushes subnormal results
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) - tol)
    return g


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 5), (2, 33), (4, 1000), (3, 8193), (2, 50021), (61, 3203)])
def test_backward(M, V, dtype):
    rng = np.random.default_rng(V)
    x = logits_(M, V, V + V % 3, dtype, seed=V, masked=0.2 if V > 30 else 0.0, offset=V % 4)
    gl, gh = rng.standard_normal(M).astype(np.float32), rng.standard_normal(M).astype(np.float32)
    check_bwd(x, targets_(M, V, V), gl, gh, 1.0)
    check_bwd(x, targets_(M, V, V), gl, None, 0.7)
    check_bwd(x, targets_(M, V, V), None, gh, 1.6)


@pytest.mark.gpu
def test_backward_in_place_strided_and_empty_rows():
    rng = np.random.default_rng(0)
    M, V = 6, 9001
    x = logits_(M, V, V + 3, "bf16", seed=4, masked=0.3)
    x[2] = -math.inf
    gl, gh = rng.standard_normal(M).astype(np.float32), rng.standard_normal(M).astype(np.float32)
    t = targets_(M, V, 0)
    # an output whose rows lie differently to 16-byte boundaries; what lies between its rows stays
    buf = torch.full((M, V + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    a = check_bwd(x, t, gl, gh, 1.0, out=buf[:, 1:V + 1])
    assert (buf[:, 0] == 5).all() and (buf[:, V + 1:] == 5).all()
    assert (a[2] == 0).all()
    inplace = x.clone(memory_format=torch.preserve_format)
    y = torch.empty(M, V + 3, dtype=torch.bfloat16, device="cuda")[:, :V]
    y.copy_(x)
    r = T.token_logprobs(x, torch.from_numpy(t).cuda())
    T.token_logprobs_backward(y, torch.from_numpy(t).cuda(), r.lse, r.entropy, torch.from_numpy(gl).cuda(),
                              torch.from_numpy(gh).cuda(), out=y)
    torch.cuda.synchronize()
    assert torch.equal(y, a) and torch.equal(inplace, x)


@pytest.mark.gpu
def test_gradient_against_differences():
    """Along a random direction the measured change of the forward's own
    outputs agrees with the gradient: step h, fp32 outputs off by about 1e-5,
    curvature h^2: 1e-5 / h + h^2 with h = 0.02 stays under 5e-3 of the scale."""
    rng = np.random.default_rng(1)
    M, V, h = 4, 501, 0.02
    x = torch.from_numpy(rng.standard_normal((M, V)).astype(np.float32) * 2).cuda()
    u = torch.from_numpy(rng.standard_normal((M, V)).astype(np.float32)).cuda()
    t = torch.from_numpy(rng.integers(0, V, M).astype(np.int32)).cuda()
    gl, gh = (torch.from_numpy(rng.standard_normal(M).astype(np.float32)).cuda() for _ in range(2))
    r = T.token_logprobs(x, t)
    g = T.token_logprobs_backward(x, t, r.lse, r.entropy, gl, gh)
    f = lambda z: (lambda q: (gl * q.logprob + gh * q.entropy).double())(T.token_logprobs(z.contiguous(), t))
    num = (f(x + h * u) - f(x - h * u)) / (2 * h)
    ana = (g.double() * u.double()).sum(1)
    assert torch.all((num - ana).abs() <= 5e-3 * (1 + ana.abs()))


@pytest.mark.gpu
def test_capture_streams_and_concurrent_calls():
    """A captured call replays on new contents; two streams at once do not
    disturb each other (no workspace is shared)."""
    M, V = 7, 33333
    x = logits_(M, V, V, "bf16", seed=8)
    t = torch.from_numpy(targets_(M, V, 3)).cuda()
    gl = torch.ones(M, device="cuda")
    T.token_logprobs(x, t, top_k=5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = T.token_logprobs(x, t, top_k=5)
        d = T.token_logprobs_backward(x, t, r.lse, r.entropy, gl, gl)
    x.copy_(logits_(M, V, V, "bf16", seed=9))
    g.replay()
    torch.cuda.synchronize()
    e = T.token_logprobs(x, t, top_k=5)
    d2 = T.token_logprobs_backward(x, t, e.lse, e.entropy, gl, gl)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(r, e)) and torch.equal(d, d2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    y = logits_(M, V, V, "bf16", seed=10)
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs.append((T.token_logprobs(x, t, top_k=5, stream=s1), T.token_logprobs(y, t, top_k=5, stream=s2)))
    torch.cuda.synchronize()
    ref = T.token_logprobs(y, t, top_k=5)
    torch.cuda.synchronize()
    for a, b in outs:
        assert all(torch.equal(p, q) for p, q in zip(a, e)) and all(torch.equal(p, q) for p, q in zip(b, ref))


def check_rows(x, t, k, scale):
    """The forward pass against 64-bit torch on the device (many long rows).
    The same tolerance as check_fwd."""
    r = T.token_logprobs(x, t, top_k=k, scale=scale)
    torch.cuda.synchronize()
    V = x.shape[1]
    ls = (4 * (math.log(V) + 1) + V / 128 + 69) * U       # a thread's share: at least 128 threads to a row
    for a in range(0, x.shape[0], 64):
        raw = x[a:a + 64].double()
        z = raw * float(np.float32(scale))
        lse = torch.logsumexp(z, 1)
        q = z - lse[:, None]
        H = -(torch.exp(q) * q.masked_fill(torch.isinf(q), 0)).sum(1)
        lp = q.gather(1, t[a:a + 64].long()[:, None])[:, 0]
        ids = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :k]
        top = q.gather(1, ids)
        big = raw.masked_fill(torch.isinf(raw), 0).abs().amax(1) * scale
        assert torch.equal(r.top_ids[a:a + 64].long(), ids)
        for got, ref, tol in ((r.logprob, lp, ls + 8 * U * (lp.abs() + 1)), (r.lse, lse, ls + 4 * U * (lse.abs() + big)),
                              (r.entropy, H, 2 * ls * (1 + math.log(V)) + 4 * U * (H.abs() + 1)),
                              (r.top_logprobs, top, ls + 8 * U * (top.abs() + 1))):
            got = got[a:a + 64].double()
            same = got == ref                              # -inf
            assert (same | ((got - ref).abs() <= tol)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,M,V,k,masked", [("bf16", 640, 140003, 8, 0.0), ("fp32", 601, 70001, 32, 0.5),
                                                ("fp16", 1200, 33000, 1, 0.9), ("bf16", 300, 140003, 20, 0.0),
                                                ("bf16", 9000, 1027, 5, 0.2)])
def test_many_long_rows(dtype, M, V, k, masked):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, V, generator=g, device="cuda") * 3
    x[torch.rand(M, V, generator=g, device="cuda") < masked] = -math.inf
    t = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    check_rows(x.to(DT[dtype]), t, k, 1.3)


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["up", "flat", "saw"])
def test_many_rows_in_order(order):
    """Rows that fill the SMs by themselves and overflow the survivor buffers."""
    V = 40007
    i = torch.arange(V, dtype=torch.float32)
    row = {"up": i / V * 20 - 10, "flat": torch.full((V,), 0.5), "saw": (i % 64) / 8}[order]
    x = row.bfloat16().expand(620, V).contiguous().cuda()
    check_rows(x, torch.arange(620, device="cuda", dtype=torch.int32), 32, 1.0)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows whose first element lies past 2^31: forward and gradient of the
    last rows, with the first rows as they were."""
    M, V = 17000, 131000
    x = torch.zeros(M, V, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    x[rows] = (torch.randn(len(rows), V, device="cuda") * 3).bfloat16()
    t = torch.full((M,), 5, device="cuda", dtype=torch.int32)
    t[rows] = torch.tensor([V - 1, 7, V // 2, 3, V - 2], device="cuda", dtype=torch.int32)
    r = T.token_logprobs(x, t, top_k=3)
    torch.cuda.synchronize()
    z = x[rows].double()
    lse = torch.logsumexp(z, 1)
    assert ((r.lse[rows].double() - lse).abs() <= 1e-5).all()
    lp = z.gather(1, t[rows].long()[:, None])[:, 0] - lse
    assert ((r.logprob[rows].double() - lp).abs() <= 2e-5).all()
    assert torch.equal(r.top_ids[rows].long(), torch.sort(z, dim=1, descending=True, stable=True).indices[:, :3])
    gl = torch.ones(M, device="cuda")
    T.token_logprobs_backward(x, t, r.lse, r.entropy, gl, out=x)
    torch.cuda.synchronize()
    ref = -torch.exp(z - lse[:, None])
    ref.scatter_add_(1, t[rows].long()[:, None], torch.ones(len(rows), 1, device="cuda", dtype=torch.float64))
    assert ((x[rows].double() - ref).abs() <= 2 ** -8 * ref.abs() * (1 + 2 ** -6) + 1e-7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [1, 3, 17, 40, 1000, 8191, 20007])
@pytest.mark.parametrize("shift", range(1, 9))
def test_backward_of_rows_that_lie_differently(dtype, V, shift):
    """Logits and gradient at every distance to each other's 16-byte
    boundaries: the same values as with equally placed rows, nothing written
    beside them."""
    g = torch.Generator(device="cuda").manual_seed(V)
    dt = DT[dtype]
    x0 = (torch.randn(3, V, generator=g, device="cuda") * 3).to(dt)
    t = torch.randint(0, V, (3,), generator=g, device="cuda", dtype=torch.int32)
    r = T.token_logprobs(x0, t)
    gl, gh = torch.randn(3, generator=g, device="cuda"), torch.randn(3, generator=g, device="cuda")
    ref = T.token_logprobs_backward(x0, t, r.lse, r.entropy, gl, gh)
    buf = torch.full((3, V + 16), math.nan, dtype=dt, device="cuda")
    x = buf[:, shift:shift + V]
    x.copy_(x0)
    out = torch.full((5, V + 3), 7.0, dtype=dt, device="cuda")
    T.token_logprobs_backward(x, t, r.lse, r.entropy, gl, gh, out=out[1:4, 1:V + 1])
    torch.cuda.synchronize()
    assert torch.equal(out[1:4, 1:V + 1], ref)
    out[1:4, 1:V + 1] = 7.0
    assert (out == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", [(3, 20011), (5, 70001), (700, 4099)])
def test_one_logit_far_above_the_others(dtype, M, V):
    """A token forced by a large bias (2^33: steps of 2^10 in fp32) takes all
    the probability, wherever it stands and whatever its thread reads after it."""
    x = logits_(M, V, V, dtype, seed=V)
    rows = torch.arange(M)
    t = (rows * 7919) % V
    t[0], t[1] = 0, V - 1
    x[rows.cuda(), t.cuda()] = 2.0 ** 33
    r = check_fwd(x, t.numpy().astype(np.int32), 5, 1.0)
    assert (r.logprob == 0).all() and (r.entropy == 0).all()


FILLS = [("bf16", f) for f in (-1e4, -1e9, -5e9, -1e10, -1e11, -1e12, -1e15, -1e20, -1e30)]
FILLS += [("fp32", f) for f in (-1e4, -1e7, -1.2e7, -1e9, -5e9, -1e10, -1e11, -1e12, -1e15, -1e20, -1e30)]
FILLS += [("fp16", f) for f in (-1e4, -65504.0)]


def filled_(M, V, dtype, fill, seed):
    """Rows masked by a finite fill: here and there, in long runs (threads that
    see nothing else, or nothing else for many tiles), all but one, throughout."""
    x = logits_(M, V, V, dtype, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for m in range(M):
        if m % 6 == 0:
            x[m][torch.rand(V, generator=gen, device="cuda") < 0.4] = fill
        elif m % 6 == 1:
            x[m, :V * 3 // 4] = fill
        elif m % 6 == 2:
            x[m, V // 4:] = fill
        elif m % 6 == 3:
            x[m, :m * 37 % V] = fill
            x[m, m * 37 % V + 1:] = fill
        elif m % 6 == 4:
            x[m] = fill
        else:
            x[m, :V - 2] = fill
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fill", FILLS)
def test_forward_masked_by_a_finite_fill(dtype, fill):
    for M, V, scale in ((6, 50021, 1.0), (12, 3001, 0.7), (606, 4099, 1.0)):
        check_fwd(filled_(M, V, dtype, fill, seed=V), targets_(M, V, M), 8, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("top", [2e7, 1e10, 1e12, 1e20, 1e30])
def test_forward_large_logits(dtype, top):
    """A forced token, two that tie, and rows that lie far up as a whole."""
    V = 30011
    x = logits_(5, V, V, dtype, seed=3)
    x[0, 17] = top
    x[1, 20000] = top
    x[2, 5] = x[2, 25000] = top
    x[3] = x[3] * (top / 4)
    x[4] = top
    t = np.array([17, 20000, 25000, 9, 8], dtype=np.int32)
    check_fwd(x, t, 6, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scale", [1e-10, 1e-8, 1e-6, 1e-3, 1e3, 1e6, 1e8, 1e10, 1e20, 1e30])
def test_forward_scales(dtype, scale):
    for M, V in ((3, 20011), (600, 2051)):
        x = logits_(M, V, V, dtype, seed=V, masked=0.1)
        x[2, 5], x[2, 1900] = x[2].max(), x[2].max()      # a tie for the first place
        check_fwd(x, targets_(M, V, M), 8, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_between_the_forms(dtype):
    """Maxima on both sides of 2^24 in units of ln 2, a few units apart, so that
    threads with either reference of their exponents meet."""
    V = 20011
    gen = torch.Generator().manual_seed(0)
    base = 2.0 ** 24 * math.log(2)
    for sign in (1.0, -1.0):
        x = sign * base + torch.randint(-8, 9, (4, V), generator=gen).double()
        x[1, 1000:] -= 6
        x[2, :15000] -= 4
        check_fwd(x.to(DT[dtype]).cuda(), targets_(4, V, 1), 4, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fill", FILLS)
def test_backward_masked_by_a_finite_fill(dtype, fill):
    """Filled logits have no gradient; a row keeps its other ones."""
    rng = np.random.default_rng(4)
    M, V = 12, 9001
    x = filled_(M, V, dtype, fill, seed=2)
    x[4::6] = x[0].clone()                                 # (rows with something left)
    gl, gh = rng.standard_normal(M).astype(np.float32), rng.standard_normal(M).astype(np.float32)
    t = np.full(M, V - 1, dtype=np.int32)
    g = check_bwd(x, t, gl, gh, 1.0)
    off = x == torch.tensor(fill, dtype=x.dtype)
    off[torch.arange(M), torch.from_numpy(t).long()] = False
    assert (g[off] == 0).all() and g.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [2e38, 3e38, 1e-38, 1e-43])
def test_forward_scales_at_the_ends_of_the_range(dtype, scale):
    """Scales whose product with log2 e is infinite or subnormal; every z is a
    finite fp32 value, every difference too."""
    V = 20011
    x = logits_(6, V, V, dtype, seed=1) * (0.02 if scale > 1 else 1e10)
    x[1] = 0
    x[2] = x[2] * (2.0 ** -124 if scale > 1 else 1e20)     # z of a few, or all alike
    x[3, 9:] = -math.inf
    x[4] = -math.inf
    x[5, ::2] = x[5, 0]
    check_fwd(x, targets_(6, V, 3), 8, scale)


def check_far_bwd(x, t, gl, gh, scale, out=None):
    """The gradient where lse is too large to tell p from: the row's own sum is
    used.  z - max is rounded twice (2 u of it), the sum adds V / 128 + 64 terms
    and expf's 4 u, its logarithm and the difference u each; p then carries
    4 u + the error of log p.  The entropy is the forward pass's (its bound)."""
    r = T.token_logprobs(x, t, scale=scale)
    g = T.token_logprobs_backward(x, t, r.lse, r.entropy, gl, gh, scale=scale, out=out)
    torch.cuda.synchronize()
    assert (r.lse.abs() >= 1024).all()
    return g


def far_reference(x, t, gl, gh, scale):
    """(gradient, its tolerance), in 64 bits."""
    z = x.double() * float(np.float32(scale))
    V = x.shape[1]
    q = torch.log_softmax(z, 1)
    p = torch.exp(q)
    safe = torch.where(p > 0, q, 0.0)
    H = -(p * safe).sum(1, keepdim=True)
    hot = torch.zeros_like(z).scatter_(1, t.clamp(min=0).long()[:, None], 1.0)
    a = torch.where(t < 0, 0.0, gl).double()[:, None]
    b = gh.double()[:, None]
    ref = scale * (a * (hot - p) - b * p * (safe + H))
    ls = (4 * (math.log(V) + 1) + V / 128 + 69) * U
    eh = 2 * ls * (1 + math.log(V)) + 4 * U * (H + 1)
    elp = ls + 4 * U * (safe.abs() + 1)
    rel = elp + 4 * U
    tol = scale * p * (a.abs() * (rel + 4 * U) + b.abs() * ((safe.abs() + H) * (rel + 4 * U) + elp + eh))
    tol = tol + scale * a.abs() * 4 * U * hot + torch.finfo(x.dtype).eps / 2 * ref.abs() * (1 + 2 ** -10)
    return ref, tol + (2.0 ** -25 if x.dtype == torch.float16 else 0.0) + scale * 2.0 ** -126


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fill", [("bf16", -1e9), ("bf16", -3e38), ("fp16", -65504.0), ("fp16", 60000.0),
                                        ("fp32", -1e4), ("fp32", -1e9), ("fp32", -1e20), ("fp32", -3.4028234e38),
                                        ("fp32", 1e12)])
@pytest.mark.parametrize("V", [1, 2, 300, 9001, 70001])
def test_backward_of_rows_far_from_zero(dtype, fill, V):
    """Rows filled throughout (uniform), filled but for one or for ten above,
    and ordinary rows among them, out of place, in place and strided."""
    M = 7
    x = torch.full((M, V + 3), fill, dtype=DT[dtype], device="cuda")[:, :V]
    gen = torch.Generator(device="cuda").manual_seed(V)
    if V > 100:
        up = torch.nextafter(torch.tensor(fill).to(DT[dtype]).float(), torch.tensor(math.inf)).item() if dtype == "fp32" \
            else float(torch.tensor(fill).to(DT[dtype])) * (1 + math.copysign(2 ** -6, fill))
        x[1, 5] = up
        x[2, 20:30] = up
        x[3, ::2] = -math.inf
    t = torch.tensor([0, min(5, V - 1), V - 1, 0, -1, V // 2, 0], dtype=torch.int32, device="cuda")
    gl, gh = (torch.randn(M, generator=gen, device="cuda") for _ in range(2))
    ref, tol = far_reference(x, t, gl, gh, 1.0)
    buf = torch.full((M + 2, V + 9), 5.0, dtype=DT[dtype], device="cuda")
    for out in (None, buf[1:M + 1, 1:V + 1], x):
        g = check_far_bwd(x, t, gl, gh, 1.0, out=out)
        assert ((g.double() - ref).abs() <= tol).all()
    buf[1:M + 1, 1:V + 1] = 5.0
    assert (buf == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scale", [1e4, 1e10])
def test_backward_at_large_scales(dtype, scale):
    V = 30011
    x = logits_(5, V, V, dtype, seed=9)
    x[2, 100:104] = x[2].max()                          # four share the probability
    t = torch.tensor([3, -1, 101, 9, V - 1], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    gl, gh = (torch.randn(5, generator=gen, device="cuda") / scale for _ in range(2))
    ref, tol = far_reference(x, t, gl, gh, scale)
    g = check_far_bwd(x, t, gl, gh, scale)
    assert ((g.double() - ref).abs() <= tol).all()


@pytest.mark.gpu
def test_backward_of_far_rows_leaves_the_others():
    """Rows on either side of the change in one call: the ordinary ones as
    without them; just below and above it both forms agree with the formula."""
    V = 20011
    x = logits_(6, V, V, "fp32", seed=5)
    t = torch.arange(6, device="cuda", dtype=torch.int32)
    gl = torch.ones(6, device="cuda")
    r = T.token_logprobs(x, t)
    plain = T.token_logprobs_backward(x, t, r.lse, r.entropy, gl, gl)
    y = x.clone()
    y[1] += 1e5
    y[4] = -1e9
    r = T.token_logprobs(y, t)
    mixed = T.token_logprobs_backward(y, t, r.lse, r.entropy, gl, gl)
    torch.cuda.synchronize()
    assert all(torch.equal(plain[i], mixed[i]) for i in (0, 2, 3, 5))
    check_bwd(x - 1000, t.cpu().numpy(), gl.cpu().numpy(), gl.cpu().numpy(), 1.0)
    check_bwd(x - 1100, t.cpu().numpy(), gl.cpu().numpy(), gl.cpu().numpy(), 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-38, 2.5e-38, 1e-37])
def test_forward_of_logits_whose_differences_are_infinite(dtype, scale):
    """Logits all over the type's range at scales that bring them to a few units."""
    for M, V in ((4, 20011), (600, 1027)):
        gen = torch.Generator().manual_seed(V)
        x = ((torch.rand(M, V, generator=gen) * 2 - 1) * 3.3e38).to(DT[dtype]).cuda()
        x[1, :900] = -3.3e38
        x[2, 7:] = torch.finfo(DT[dtype]).min
        check_fwd(x, targets_(M, V, 1), 6, scale)


@pytest.mark.gpu
def test_torch_api_refuses_outputs_that_do_not_fit():
    """What is missing among the given outputs is refused as the library refuses it."""
    x = logits_(3, 100, 100, "bf16", seed=3)
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    f = torch.empty(3, device="cuda")
    ids, top = torch.empty((3, 2), dtype=torch.int32, device="cuda"), torch.empty((3, 2), device="cuda")
    for out, k, targets in ((T.TokenLogprobs(f, None, None, None, None), 2, t), (T.TokenLogprobs(f, None, None, ids, None), 2, t),
                            (T.TokenLogprobs(None, None, None, None, None), 0, t), (T.TokenLogprobs(f, None, None, None, None), 0, None),
                            (T.TokenLogprobs(f, f, None, None, None), 0, t)):
        with pytest.raises(fnb.FnError):
            T.token_logprobs(x, targets, top_k=k, out=out)
    with pytest.raises(ValueError):
        T.token_logprobs(x, t, top_k=3, out=T.TokenLogprobs(f, None, None, ids, top))
    r = T.token_logprobs(x, t, top_k=2, out=T.TokenLogprobs(None, f, None, ids, top))
    ref = T.token_logprobs(x, t, top_k=2)
    torch.cuda.synchronize()
    assert torch.equal(r.entropy, ref.entropy) and torch.equal(ids, ref.top_ids) and torch.equal(top, ref.top_logprobs)
