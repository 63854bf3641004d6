"""moe_linear_q4, moe_sample and moe_balance_loss against plain references in 64 bits.

Tolerances:
  linear, exact cases   bits: inputs are small whole numbers and scales powers of two, so every partial sum of any
                        order is a whole multiple of one unit below 2^24 units and fp32 holds it exactly
  linear, other cases   a sum passes through at most 2 * 128 roundings inside a group (products with the code and the
                        correction by 8), K/32 of the groups' sums and 8 more (scale, bias, waves), each of at most
                        2^-23 (a matrix instruction may cut off) of a partial sum, which stays below the sum of
                        |x| * scale * (code + 8); bf16 outputs add half a step, 2^-8, of the value
  sample                ids equal; prob one rounding of a double (2^-24) and 2^-S per id of the row's mass
  balance               counts equal; shares are sums of doubles: (T + E + 64) * 2^-52 relative; lse and loss one
                        rounding to fp32 of those; gradients: below
"""
import numpy as np
import pytest

import ops_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_vram_slot_amd as mod
    mod.lib()
    return mod


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def code(m, name):
    return m.MOE_X_BF16 if name == "bf16" else m.MOE_X_F32


def host64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ linear


def linear(m, x, wq, scales, group, bias, yt, ldx=None, ldy=None, stream=None):
    """moe_linear_q4 on padded copies; the padding of y must stay as it was."""
    T, K = x.shape
    N = wq.shape[0]
    ldx, ldy = ldx or K, ldy or N
    xp = torch.full((T, ldx), float("nan"), dtype=x.dtype, device="cuda")
    xp[:, :K] = x
    y = torch.full((T + 1, ldy), 77.0, dtype=DT[yt], device="cuda")
    m.moe_linear_q4(xp, code(m, "bf16" if x.dtype == torch.bfloat16 else "f32"), ldx, wq, scales, group, bias, T, N, K, y,
                    code(m, yt), ldy, stream)
    torch.cuda.synchronize()
    assert torch.all(y[T] == 77.0) and torch.all(y[:, N:] == 77.0)
    return y[:T, :N]


def weights(N, K, group, seed, power_of_two=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wq = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    if power_of_two:
        scales = torch.pow(2.0, -torch.randint(0, 3, (N, K // group), device="cuda", generator=g).float()).half()
    else:
        scales = (0.003 + 0.004 * torch.rand(N, K // group, device="cuda", generator=g)).half()
    return wq, scales, g


SHAPES = [(1, 1, 32, 32), (1, 3, 96, 32), (2, 16, 128, 128), (3, 17, 64, 64), (4, 63, 160, 32), (5, 257, 1056, 32),
          (8, 33, 192, 64), (15, 100, 256, 128), (16, 64, 512, 64), (17, 65, 1088, 64), (31, 130, 384, 128),
          (33, 48, 2048, 32), (64, 300, 640, 128), (65, 129, 128, 32), (130, 31, 1536, 64), (1, 2048, 2048, 32),
          (300, 70, 256, 32), (7, 1, 8192, 128), (1, 5000, 4096, 128),
          # many rows by many tokens, in whole tiles and past them
          (40, 32769, 128, 32), (64, 33000, 384, 128), (65, 16400, 160, 32), (130, 11000, 448, 64), (33, 32800, 1088, 64),
          (20, 32777, 192, 64), (300, 7000, 96, 32), (64, 80000, 320, 32),
          # rows of x too long to lie in LDS whole
          (16, 64, 8192, 128), (13, 40, 8224, 32), (40, 100, 8256, 64), (3, 50, 8224, 32), (8, 5000, 4128, 32),
          (23, 2000, 4160, 64), (64, 4099, 2048, 32), (33, 70, 2080, 32), (4, 300, 12320, 32), (7, 333, 8064, 64),
          (1, 37, 40000, 64)]


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K,group", SHAPES)
def test_linear_exact(m, T, N, K, group, xt):
    # |x| <= 2, K * 23 * 2 < 2^21, scales 1, 1/2, 1/4 (units of 1/4): below 2^24 units
    wq, scales, g = weights(N, K, group, T * 1000 + N, True)
    x = torch.randint(-2, 3, (T, K), device="cuda", generator=g).to(DT[xt])
    bias = torch.randint(-8, 9, (N,), device="cuda", generator=g).float() if N % 2 else None
    want, _ = ref.linear_q4(host64(x), wq.cpu().numpy(), scales.cpu().numpy(), group, None if bias is None else host64(bias))
    got = linear(m, x, wq, scales, group, bias, "f32", ldx=K + 8 if T > 1 else K, ldy=N + 3)
    np.testing.assert_array_equal(host64(got), want)
    got = linear(m, x, wq, scales, group, bias, "bf16", ldy=N + 1)
    np.testing.assert_array_equal(host64(got), host64(torch.from_numpy(want).float().to(torch.bfloat16)))


@pytest.mark.parametrize("T", [1, 3, 16, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_every_weight_by_itself(m, T, group):
    """One input of a token is not zero: its outputs are one column of the weights, with all 20 bits of an fp32 x."""
    N, K = 37, 512
    wq, scales, g = weights(N, K, group, group, True)
    q, d = ref.codes(wq.cpu().numpy()).astype(np.float64) - 8, np.repeat(scales.double().cpu().numpy(), group, axis=1)
    for k0 in range(0, K, 4 * T):
        ks = (k0 + np.arange(T) * 5) % K
        for xt, bits in (("f32", 20), ("bf16", 8)):
            v = torch.randint(1 << (bits - 1), 1 << bits, (T,), device="cuda", generator=g)
            x = torch.zeros(T, K, device="cuda")
            x[torch.arange(T), torch.from_numpy(ks).cuda()] = v.float()
            got = linear(m, x.to(DT[xt]), wq, scales, group, None, "f32")
            np.testing.assert_array_equal(host64(got), (host64(v)[None] * (q * d)[:, ks]).T)


@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,N,K,group", SHAPES + [(1, 40000, 2048, 32), (20, 6000, 4096, 128)])
def test_linear_random(m, T, N, K, group, xt, yt):
    wq, scales, g = weights(N, K, group, T + N + K)
    x = torch.randn(T, K, device="cuda", generator=g).to(DT[xt])
    bias = torch.randn(N, device="cuda", generator=g) if N % 2 == 0 else None
    want, size = ref.linear_q4(host64(x), wq.cpu().numpy(), scales.cpu().numpy(), group, None if bias is None else host64(bias))
    got = host64(linear(m, x, wq, scales, group, bias, yt, ldx=K + 16))
    tol = (2 * 128 + K / 32 + 8) * 2.0 ** -23 * size
    assert np.all(np.abs(got - want) <= tol + (2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) if yt == "bf16" else 0))
    # roundings of either sign: over all outputs the root mean square stays far below the worst case.  Each of the
    # about 34 roundings that a block of 32 takes is at most 2^-24 of sums of size 12 * sqrt(32) * d * |x| (codes 0..15
    # and the correction, random signs of x) against outputs of 4.6 * sqrt(32) * d * |x| a block: below
    # sqrt(34) * 2.6 * 2^-24 = 9e-7 relative, and the blocks' sums add sqrt(K / 32) * 2^-24 at most (K = 8192: 1e-6)
    if yt == "f32" and want.size >= 1000:
        assert np.linalg.norm(got - want) <= 2e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("T,N,K,group", [(1, 37, 512, 128), (8, 100, 1024, 64), (16, 64, 512, 32), (64, 32800, 256, 128)])
def test_linear_scales_aligned_to_their_elements_alone(m, T, N, K, group):
    wq, scales, g = weights(N, K, group, T + N, True)
    x = torch.randint(-2, 3, (T, K), device="cuda", generator=g).bfloat16()
    moved = torch.empty(scales.numel() + 1, dtype=torch.float16, device="cuda")[1:].view_as(scales)
    moved.copy_(scales)
    assert moved.data_ptr() % 4 == 2
    assert torch.equal(linear(m, x, wq, moved, group, None, "f32"), linear(m, x, wq, scales, group, None, "f32"))


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K,group", [(1, 300, 512, 64), (7, 300, 512, 64), (24, 300, 1024, 32), (20, 66000, 256, 128),
                                         (40, 33000, 256, 32)])
def test_linear_scales_with_its_input(m, T, N, K, group, xt):
    """Powers of two go through every rounding, 90 up and down, in all 24 bits of an fp32 x."""
    wq, scales, g = weights(N, K, group, N + K)
    x = torch.randn(T, K, device="cuda", generator=g).to(DT[xt])
    x = torch.where(x.abs() < 2.0 ** -10, torch.ones_like(x), x)  # the smallest bit of x times 2^-90: 2^-123
    want = linear(m, x, wq, scales, group, None, "f32")
    for s in (2.0 ** 90, 2.0 ** -90):
        assert torch.equal(linear(m, x * s, wq, scales, group, None, "f32"), want * s)


@pytest.mark.parametrize("N", [200, 66000])
def test_linear_bits_do_not_depend_on_other_tokens(m, N):
    wq, scales, g = weights(N, 1024, 32, 5)
    x = torch.randn(24, 1024, device="cuda", generator=g).bfloat16()
    a = linear(m, x, wq, scales, 32, None, "f32")
    x2 = x.clone()
    x2[3], x2[17] = float("nan"), float("inf")
    x2[20:] = 3.0
    b = linear(m, x2, wq, scales, 32, None, "f32")
    keep = [t for t in range(20) if t not in (3, 17)]
    assert torch.equal(a[keep], b[keep])
    assert torch.equal(a, linear(m, x, wq, scales, 32, None, "f32"))
    assert not torch.any(torch.isfinite(b[3])) and not torch.any(torch.isfinite(b[17]))


@pytest.mark.parametrize("T", [2, 40])
def test_linear_offsets_past_32_bits(m, T):
    """Codes past 4 GiB: the last rows of a tall matrix."""
    N, K, group = (1 << 20) + 70000, 8192, 128  # 4.58 GB of codes
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB of device memory")
    wq = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.ones(N, K // group, dtype=torch.float16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.tensor([0, 1, (1 << 20) - 1, 1 << 20, (1 << 20) + 5, N - 2, N - 1], device="cuda")
    wq[rows] = torch.randint(0, 256, (7, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    x = torch.randint(-1, 2, (T, K), device="cuda", generator=g).bfloat16()
    y = torch.empty(T, N, device="cuda")
    m.moe_linear_q4(x, m.MOE_X_BF16, K, wq, scales, group, None, T, N, K, y, m.MOE_X_F32, N)
    want, _ = ref.linear_q4(host64(x), wq[rows].cpu().numpy(), scales[rows].cpu().numpy(), group)
    np.testing.assert_array_equal(host64(y[:, rows]), want)
    zero = -8.0 * x.float().sum(dim=1, keepdim=True)
    assert torch.all(y[:, 2:(1 << 20) - 1] == zero)


@pytest.mark.parametrize("T,N", [(8, 100), (16, 100), (34, 100), (40, 33000)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_linear_rows_past_32_bits(m, T, N, xt):
    """Tokens and outputs 2^26 values apart and more: the last start past 2^31 bytes, or values."""
    K, group = 256, 64
    ld = (1 << 31) // (T - 1) // 8 * 8 + 8
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of device memory")
    wq, scales, g = weights(N, K, group, T)
    x = torch.randn(T, K, device="cuda", generator=g).to(DT[xt])
    far = torch.empty((T - 1) * ld + K, dtype=DT[xt], device="cuda")
    y = torch.empty((T - 1) * ld + N, device="cuda")
    torch.as_strided(far, (T, K), (ld, 1)).copy_(x)
    m.moe_linear_q4(far, code(m, xt), ld, wq, scales, group, None, T, N, K, y, m.MOE_X_F32, ld)
    assert torch.equal(torch.as_strided(y, (T, N), (ld, 1)), linear(m, x, wq, scales, group, None, "f32"))


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K,group", [(513, 700, 256, 64), (4097, 300, 288, 32), (8193, 520, 256, 128), (1 << 20, 3, 32, 32)])
def test_linear_prompts(m, T, N, K, group, xt):
    """Whole numbers, as in test_linear_exact, by as many tokens as a prompt has, and by as many as a call takes."""
    wq, scales, g = weights(N, K, group, T + N, True)
    x = torch.randint(-2, 3, (T, K), device="cuda", generator=g).to(DT[xt])
    want, _ = ref.linear_q4(host64(x), wq.cpu().numpy(), scales.cpu().numpy(), group)
    np.testing.assert_array_equal(host64(linear(m, x, wq, scales, group, None, "f32")), want)


# ------------------------------------------------------------------ sample


def draw(m, l, u, temperature=None, min_p=None, top_k=None, top_p=None, ldl=None, with_prob=True):
    """moe_sample on a padded copy of l [T][V] (the padding would win every draw)."""
    T, V = l.shape
    ldl = ldl or V
    lp = torch.full((T, ldl), 1e4, dtype=l.dtype, device="cuda")
    lp[:, :V] = l
    ids = torch.full((T + 1,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((T + 1,), -9.0, device="cuda") if with_prob else None
    n = m.moe_sample_workspace_bytes(T, V)
    ws = torch.randint(0, 256, (n + 64,), dtype=torch.uint8, device="cuda")  # needs no clearing
    tail = ws[n:].clone()
    m.moe_sample(lp, code(m, "bf16" if l.dtype == torch.bfloat16 else "f32"), ldl, T, V, temperature, min_p, top_k, top_p,
                 u, ids, prob, ws, n)
    torch.cuda.synchronize()
    assert int(ids[T]) == -9 and torch.equal(ws[n:], tail)
    if not with_prob:
        return ids[:T].cpu().numpy(), None
    assert float(prob[T]) == -9.0
    return ids[:T].cpu().numpy(), host64(prob[:T])


def check_draw(m, l, u, temperature=None, min_p=None, top_k=None, top_p=None, ldl=None):
    ids, prob = draw(m, l, u, temperature, min_p, top_k, top_p, ldl)
    lh, uh = host64(l), host64(u)
    opt = [None if a is None else a.double().cpu().numpy() for a in (temperature, min_p, top_k, top_p)]
    V = l.shape[1]
    for t in range(l.shape[0]):
        a = [d if o is None else o[t] for o, d in zip(opt, (1.0, 0.0, 0, 1.0))]
        want, p, _ = ref.sample_row(lh[t], uh[t], a[0], a[1], int(a[2]), a[3])
        assert ids[t] == want, f"row {t}: {ids[t]}, not {want} ({a}, u {uh[t]})"
        # rounding to fp32, and whole multiples of 2^-S (S = 62 - ceil(log2 V), 51 at most), half a step for each id of a
        # mass of 1 or more
        assert abs(prob[t] - p) <= 2.0 ** -24 * p + V * 2.0 ** -min(51, 62 - max(V - 1, 0).bit_length()) + 1e-38


def settings(T, g, kind, V):
    r = torch.rand(5, T, device="cuda", generator=g)
    temperature = 0.3 + 1.5 * r[0]
    if kind == "none":
        return None, None, None, None
    if kind == "temperature":
        return temperature, None, None, None
    k = (1 + r[1] * min(V, 100)).to(torch.int32)
    p, q = 0.02 + 0.97 * r[2], 0.001 + 0.2 * r[3]
    if kind == "k":
        return temperature, None, k, None
    if kind == "p":
        return temperature, None, None, p
    if kind == "min":
        return temperature, q, None, None
    if kind == "wide":  # large k, the boundaries in the bulk
        return 4.0 * temperature, None, (V * (0.2 + 0.8 * r[4])).to(torch.int32), 0.5 + 0.5 * p
    row = torch.arange(T, device="cuda")
    off = lambda a, n, v: torch.where(row % n == 0, torch.full_like(a, v), a)  # noqa: E731
    return off(temperature, 5, 0), off(q, 2, 0), off(k, 3, 0), off(p, 4, 1)


@pytest.mark.parametrize("kind", ["none", "temperature", "k", "p", "min", "wide", "mixed"])
@pytest.mark.parametrize("T,V,lt", [(5, 1, "f32"), (9, 2, "bf16"), (7, 63, "f32"), (6, 1000, "bf16"), (4, 1025, "f32"),
                                    (3, 4096, "f32"), (5, 4097, "bf16"), (3, 8192, "f32"), (2, 16385, "f32"),
                                    (4, 32769, "f32"), (3, 65537, "bf16"), (2, 131072, "f32"), (1, 150001, "f32"),
                                    (40, 20011, "f32")])
def test_sample_matches_reference(m, T, V, lt, kind):
    g = torch.Generator(device="cuda").manual_seed(T * V + len(kind))
    l = (2.5 * torch.randn(T, V, device="cuda", generator=g)).to(DT[lt])
    u = torch.rand(T, device="cuda", generator=g)
    check_draw(m, l, u, *settings(T, g, kind, V), ldl=V + (3 if V % 2 else 0))


@pytest.mark.parametrize("V", [1, 7, 1000, 4500, 33000])
@pytest.mark.parametrize("levels", [1, 2, 5])
def test_sample_ties(m, V, levels):
    """Rows of a few distinct values: every boundary falls among equal logits, and ids decide."""
    T = 8
    g = torch.Generator(device="cuda").manual_seed(V + levels)
    l = torch.randint(0, levels, (T, V), device="cuda", generator=g).float() * 0.75 - 0.5
    l[1] = torch.where(l[1] == -0.5, torch.tensor(0.0, device="cuda"), l[1])
    l[1, ::2] = torch.where(l[1, ::2] == 0, torch.tensor(-0.0, device="cuda"), l[1, ::2])  # -0 and 0 are equal
    u = torch.rand(T, device="cuda", generator=g)
    check_draw(m, l, u)
    check_draw(m, l, u, top_k=torch.randint(1, V + 2, (T,), device="cuda", generator=g).to(torch.int32))
    check_draw(m, l, u, top_p=torch.rand(T, device="cuda", generator=g))
    check_draw(m, l, u, None, torch.full((T,), 0.5, device="cuda"),
               torch.randint(1, V + 2, (T,), device="cuda", generator=g).to(torch.int32),
               torch.rand(T, device="cuda", generator=g))
    check_draw(m, l, u, torch.zeros(T, device="cuda"))


@pytest.mark.parametrize("V", [6, 3000, 40000])
def test_sample_masked_and_special_rows(m, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    inf, nan = float("inf"), float("nan")
    l = torch.randn(9, V, device="cuda", generator=g)
    l[0] = -inf                                   # nothing left
    l[1] = nan                                    # nothing left
    l[2, :] = -inf
    l[2, V - 1] = -3e38                           # one candidate, near the type's lowest value
    l[3, ::2] = -inf
    l[4, ::2] = nan
    l[5, 1], l[5, V // 2] = inf, inf              # two share everything
    l[6] = torch.finfo(torch.float32).min         # a mask of the lowest value, everywhere
    l[7] = torch.finfo(torch.float32).min
    l[7, V // 3] = 1.0
    l[8] = torch.where(torch.rand(V, device="cuda", generator=g) < 0.5, 1e-45, -1e-45)  # below the normal range
    u = torch.rand(9, device="cuda", generator=g)
    one = torch.ones(9, device="cuda")
    for lt in (torch.float32, torch.bfloat16):
        x = l.to(lt)
        check_draw(m, x, u)
        check_draw(m, x, u, 0 * one)
        check_draw(m, x, u, 0.7 * one, 0.1 * one, (2 * one).to(torch.int32), 0.9 * one)
        check_draw(m, x, u, 1.3 * one, None, (max(V - 1, 1) * one).to(torch.int32), 0.5 * one)
        check_draw(m, x, u, None, 0.3 * one)


@pytest.mark.parametrize("V", [50, 5000, 50000])
def test_sample_ends_of_the_settings(m, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    T = 6
    l = 2 * torch.randn(T, V, device="cuda", generator=g)
    u = torch.rand(T, device="cuda", generator=g)
    f = lambda *v: torch.tensor(v, device="cuda")  # noqa: E731
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    inf, nan = float("inf"), float("nan")
    check_draw(m, l, u, f(-1.0, nan, 1e-30, 1e-45, 1e30, inf))
    check_draw(m, l, u, None, f(0.0, -1.0, nan, 1.0, 7.0, 1e-30))
    check_draw(m, l, u, None, None, i(-5, 0, 1, V - 1, V, 2 ** 31 - 1))
    check_draw(m, l, u, None, None, None, f(0.0, -2.0, nan, 1.0, 3.0, 1e-30))
    check_draw(m, l, u, None, None, None, f(1 - 2.0 ** -24, 1 - 2.0 ** -12, 0.5, 1e-3, inf, -inf))
    check_draw(m, l, f(0.0, 1 - 2.0 ** -24, 1e-30, nan, -0.0, -1.0))
    ids, prob = draw(m, l, f(1.0, 2.0, inf, 0.5, 0.5, 0.5))  # from 1 on: the last id that has mass
    assert list(ids[:3]) == [V - 1] * 3
    a, p = draw(m, l, u, with_prob=False)
    assert p is None and list(a) == list(draw(m, l, u)[0])


def test_sample_offsets_past_32_bits(m):
    V, ldl, T = 1000, 1 << 26, 40  # rows 2^26 values apart: the last starts past 2^31 values
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB of device memory")
    buf = torch.zeros(T * ldl - ldl + V, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn(T, V, device="cuda", generator=g).bfloat16()
    torch.as_strided(buf, (T, V), (ldl, 1)).copy_(l)
    u = torch.rand(T, device="cuda", generator=g)
    ids = torch.empty(T, dtype=torch.int32, device="cuda")
    n = m.moe_sample_workspace_bytes(T, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    m.moe_sample(buf, m.MOE_X_BF16, ldl, T, V, None, None, None, None, u, ids, None, ws, n)
    np.testing.assert_array_equal(ids.cpu().numpy(), draw(m, l, u)[0])


def test_sample_largest_vocabulary(m):
    g = torch.Generator(device="cuda").manual_seed(2)
    V = 1 << 20
    l = 2 * torch.randn(2, V, device="cuda", generator=g)
    u = torch.rand(2, device="cuda", generator=g)
    one = torch.ones(2, device="cuda")
    check_draw(m, l, u)
    check_draw(m, l, u, one, None, (300 * one).to(torch.int32), 0.9 * one)
    check_draw(m, l, u, 3 * one, 1e-4 * one, None, 0.7 * one)


@pytest.mark.parametrize("kind", ["none", "min", "k", "p", "wide", "mixed"])
@pytest.mark.parametrize("T,V,lt", [(600, 33001, "bf16"), (600, 33001, "f32"), (2000, 33001, "f32"), (2001, 20479, "bf16"),
                                    (65535, 8193, "bf16")])
def test_sample_many_long_rows(m, T, V, lt, kind):
    """More than 16384 segments of 1024 ids: a wave takes several of a row, the row's last wave fewer.  The first row of
    each setting, the last and some between are looked at, and that no row lacks its id."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    l = torch.randn(T, V, device="cuda", generator=g, dtype=DT[lt]) * 2.5
    u = torch.rand(T, device="cuda", generator=g)
    opt = settings(T, g, kind, V)
    ids, prob = draw(m, l, u, *opt, ldl=V + 1)
    assert ids.min() >= 0 and ids.max() < V and prob.min() > 0
    rows = list(range(12)) + [T // 2 + 60 * i + i for i in range(4)] + [T - 1]
    one = lambda a, t: None if a is None else a[t:t + 1]  # noqa: E731
    for t in rows:
        o = [None if a is None else float(a[t]) for a in opt]
        a = [d if v is None else v for v, d in zip(o, (1.0, 0.0, 0, 1.0))]
        want, p, _ = ref.sample_row(host64(l[t]), float(u[t]), a[0], a[1], int(a[2]), a[3])
        assert ids[t] == want, f"row {t}: {ids[t]}, not {want} ({a})"
        assert abs(prob[t] - p) <= 2.0 ** -24 * p + V * 2.0 ** -min(51, 62 - (V - 1).bit_length()) + 1e-38
        # the row alone, a segment a wave
        alone = draw(m, l[t:t + 1], u[t:t + 1], *[one(x, t) for x in opt])
        assert alone[0][0] == ids[t] and alone[1][0] == prob[t]


@pytest.mark.parametrize("V", [40, 3000, 40000])
def test_sample_signalling_nan(m, V):
    """NaN of either kind and sign is never drawn."""
    g = torch.Generator(device="cuda").manual_seed(V)
    l = torch.randn(6, V, device="cuda", generator=g)
    u = torch.rand(6, device="cuda", generator=g)
    for lt, bits in (("f32", (0x7F800001, 0x7FC00000, -0x7FFFFF, -1)), ("bf16", (0x7F81, 0x7FC0, -0x7F, -1))):
        x = l.to(DT[lt])
        raw = x.view(torch.int32 if lt == "f32" else torch.int16)
        for r, b in enumerate(bits):
            raw[r, ::2] = b
        raw[4] = bits[0]
        raw[4, V // 2] = x[5].view(raw.dtype)[0]
        check_draw(m, x, u)
        check_draw(m, x, u, torch.full((6,), 0.9, device="cuda"), None, torch.full((6,), 7, dtype=torch.int32, device="cuda"),
                   torch.full((6,), 0.8, device="cuda"))
        check_draw(m, x, u, torch.zeros(6, device="cuda"))


# ------------------------------------------------------------------ balance


def run_balance(m, z, ids, mask=None, dloss=(0.7, 0.2)):
    T, E = z.shape
    k = ids.shape[1]
    dev = dict(device="cuda")
    o = dict(counts=torch.full((E + 1,), -9, dtype=torch.int32, **dev), totals=torch.empty(2, dtype=torch.int32, **dev),
             share=torch.empty(E, dtype=torch.float64, **dev), lse=torch.full((T + 1,), -9.0, **dev),
             loss=torch.empty(2, **dev), dz=torch.full((T + 1, E), 77.0, dtype=z.dtype, **dev))
    n = m.moe_balance_workspace_bytes(T, E)
    ws = torch.randint(0, 256, (n + 64,), dtype=torch.uint8, **dev)
    tail = ws[n:].clone()
    zt = code(m, "bf16" if z.dtype == torch.bfloat16 else "f32")
    m.moe_balance_loss(z, zt, ids, mask, T, E, k, o["counts"], o["totals"], o["share"], o["lse"], o["loss"], ws, n)
    m.moe_balance_loss_bwd(z, zt, o["lse"], mask, o["counts"], o["totals"], torch.tensor(dloss, **dev), T, E, o["dz"])
    torch.cuda.synchronize()
    assert torch.equal(ws[n:], tail) and int(o["counts"][E]) == -9 and float(o["lse"][T]) == -9.0
    assert torch.all(o["dz"][T] == 77.0)
    return {k_: v[:T] if k_ in ("lse", "dz") else v[:E] if k_ == "counts" else v for k_, v in o.items()}


def check_balance(m, z, ids, mask=None, dloss=(0.7, 0.2)):
    o = run_balance(m, z, ids, mask, dloss)
    T, E = z.shape
    zh, ih = host64(z), ids.cpu().numpy()
    mh = None if mask is None else mask.cpu().numpy()
    w = ref.balance(zh, ih, mh)
    np.testing.assert_array_equal(o["counts"].cpu().numpy(), w["counts"])
    np.testing.assert_array_equal(o["totals"].cpu().numpy(), w["totals"])
    eps = (T + E + 64) * 2.0 ** -52
    assert np.all(np.abs(host64(o["share"]) - w["share"]) <= eps * w["share"] + 1e-300)
    for name in ("lse", "loss"):
        assert np.all(np.abs(host64(o[name]) - w[name]) <= (2.0 ** -24 + 2 * eps) * np.abs(w[name]) + eps), name
    # gradient: p = exp(z - lse) in fp32 from an lse rounded to fp32: relative error 2^-24 * (|lse| + |z - lse|) and 8
    # roundings of the exponential and the products; the inner sum adds E + 8 roundings of sum p |f'|, f' = f less its
    # mean, and that relative error again; bf16 outputs half a step
    n, picks = max(int(w["totals"][0]), 1), max(int(w["totals"][1]), 1)
    want = ref.balance_grad(zh, ih, np.array(dloss), mh)
    f = (w["counts"] / picks - (1 / E if int(w["totals"][1]) else 0)) * dloss[0] * E / n
    with np.errstate(invalid="ignore"):
        gap = np.where(w["p"] > 0, np.abs(zh - w["lse"][:, None]), 0)
    rel = 2.0 ** -24 * (np.abs(w["lse"])[:, None] + gap + 8)
    inner = (w["p"] * np.abs(f) * (rel + (E + 8) * 2.0 ** -24)).sum(axis=1, keepdims=True)
    zterm = np.abs(2 * dloss[1] * w["lse"])[:, None] / n
    size = np.abs(f)[None] + (w["p"] * np.abs(f)).sum(axis=1, keepdims=True) + zterm
    tol = w["p"] * (inner + size * rel * 2) + 1e-37
    # the reference subtracts f itself, not f less its mean: E + 8 roundings of doubles of the size of f and sum p f (with
    # as many picks on every expert the gradient is 0, and the reference's own rounding, 2^-52 of f, is all there is)
    raw = w["counts"] / picks * abs(dloss[0]) * E / n
    tol = tol + (E + 8) * 2.0 ** -52 * w["p"] * (raw[None] + (w["p"] * raw).sum(axis=1, keepdims=True) + zterm)
    if z.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(host64(o["dz"]) - want) <= tol)
    return o, w


def logits(T, E, seed, zt="f32", scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (scale * torch.randn(T, E, device="cuda", generator=g) + torch.randn(E, device="cuda", generator=g)).to(DT[zt])
    return z, g


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 64, 8), (16, 65, 6), (33, 127, 3), (64, 128, 8),
                                   (100, 129, 10), (257, 288, 8), (500, 512, 10), (130, 513, 4), (40, 1024, 32),
                                   (20, 1500, 7), (9, 2049, 32), (5, 4096, 2), (5003, 40, 4), (3000, 256, 8)])
def test_balance_matches_reference(m, T, E, k, zt):
    z, g = logits(T, E, T + E, zt)
    ids = z.float().topk(k, dim=1).indices.to(torch.int32).contiguous()
    check_balance(m, z, ids)
    mask = (torch.rand(T, device="cuda", generator=g) < 0.7).to(torch.uint8) * 3  # any number but 0 counts
    check_balance(m, z, ids, mask, (-1.5, 0.0))
    check_balance(m, z, ids, mask, (0.0, 2.0))


def test_balance_larger_batch(m):
    z, g = logits(20001, 96, 4)
    ids = torch.randint(-2, 99, (20001, 6), device="cuda", generator=g).to(torch.int32)  # ids out of range are left out
    check_balance(m, z, ids)


def test_balance_nothing_counted(m):
    z, g = logits(50, 32, 1)
    ids = torch.zeros(50, 4, dtype=torch.int32, device="cuda")
    for zz, ii, mask in ((z, ids, torch.zeros(50, dtype=torch.uint8, device="cuda")), (z[:0], ids[:0], None),
                         (torch.full_like(z, -float("inf")), ids, None)):
        o, _ = check_balance(m, zz, ii, mask)
        assert torch.all(o["loss"] == 0) and torch.all(o["dz"] == 0) and torch.all(o["totals"] == 0)
    # picks all out of range: shares and z loss stay, the balance loss and its gradient are 0
    o, _ = check_balance(m, z, ids - 1, None, (1.0, 0.0))
    assert float(o["loss"][0]) == 0 and float(o["loss"][1]) > 0 and torch.all(o["dz"] == 0)


def test_balance_masked_and_special_rows(m):
    inf, nan = float("inf"), float("nan")
    for zt in ("f32", "bf16"):
        z, g = logits(40, 70, 9, zt)
        ids = torch.randint(0, 70, (40, 3), device="cuda", generator=g).to(torch.int32)
        mask = torch.ones(40, dtype=torch.uint8, device="cuda")
        mask[[2, 5, 39]] = 0
        z[2], z[5, 3], z[39] = nan, inf, -inf   # masked: not looked at
        z[7] = -inf                             # nothing left: as if masked
        z[8, 1:] = -inf                         # one expert left
        z[9, ::2] = -inf
        z[10] = torch.finfo(DT[zt]).min         # a mask of the lowest value, everywhere
        z[10, 4] = 1.0
        z[11] = 80.0
        z[12] = -80.0
        check_balance(m, z, ids, mask)
        z[20, 3] = nan                          # a live NaN is not hidden
        o = run_balance(m, z, ids, mask)
        assert torch.isnan(o["loss"]).all() and torch.isnan(o["lse"][20]) and torch.isnan(o["share"]).all()
        z[20] = nan
        assert torch.isnan(run_balance(m, z, ids, mask)["loss"]).all()


def test_balance_gradient_against_differences(m):
    """dz against central differences of the operator's own losses (fp32: rounding 2^-24 * loss / h, loss below 8;
    truncation h^2 / 6 times a third derivative below 8)."""
    z, g = logits(3, 5, 2)
    ids = z.topk(2, dim=1).indices.to(torch.int32)
    h = 2.0 ** -6
    o = run_balance(m, z, ids, None, (0.8, 0.3))
    tol = 2.0 ** -24 * 8 / h + h * h / 6 * 8
    for t in range(3):
        for e in range(5):
            d = []
            for s in (h, -h):
                zz = z.clone()
                zz[t, e] += s
                d.append(host64(run_balance(m, zz, ids)["loss"]))
            want = (d[0] - d[1]) @ np.array([0.8, 0.3]) / (2 * h)
            assert abs(float(o["dz"][t, e]) - want) <= tol


def check_balance_grad(z, o, dloss, mask=None):
    """dz of fp32 softmaxes against the formula in double, from the logits themselves.

    In units of u = 2^-24: an exponential is off by |z - max| (the difference is rounded) and 2 (its own last bit); a sum
    of a row by that of its terms and D = E / 64 + 8 roundings; the division by it by 5, a product by 1.  f less its mean
    is rounded once, lse, its factor and their product once each, the two sums inside the bracket once each."""
    zh = host64(z)
    E = zh.shape[1]
    w = ref.balance(zh, np.zeros((len(zh), 1), np.int32), None if mask is None else mask.cpu().numpy())
    counts, (n, picks) = o["counts"].cpu().numpy().astype(np.float64), o["totals"].cpu().numpy().astype(np.float64)
    p, live = w["p"], w["live"]
    f = (counts * E - picks) * dloss[0] / (n * picks)
    zt = 2 * dloss[1] * w["lse"][:, None] / n
    want = p * (f[None] - (p @ f)[:, None] + zt)
    u, D = 2.0 ** -24, E / 64 + 8
    with np.errstate(invalid="ignore"):
        e = np.where(p > 0, zh.max(axis=1, keepdims=True) - zh, 0) + 2
    total = (p * e).sum(axis=1, keepdims=True) + D
    dot, size = (p * np.abs(f)).sum(axis=1, keepdims=True), np.abs(f)[None] + np.abs(zt)
    inner = (p * np.abs(f) * e).sum(axis=1, keepdims=True) + dot * (1 + D + total + 6)
    tol = p * (np.abs(f)[None] + inner + 3 * np.abs(zt) + (size + dot) * (2 + e + total + 7)) * u * (1 + 2.0 ** -10)
    tol = tol + 2.0 ** -126 * (size + dot + 1)
    if z.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    got = host64(o["dz"])
    assert np.all(np.abs(got - want)[live] <= tol[live])
    assert np.all(got[~live] == 0)


@pytest.mark.parametrize("zt,shift", [("f32", 0.0), ("f32", 1e4), ("f32", -1e6), ("f32", 1e6), ("bf16", 1e6),
                                      ("f32", 1e9), ("f32", -2e38), ("bf16", -1e30)])
@pytest.mark.parametrize("T,E,k", [(33, 64, 4), (257, 288, 8), (40, 1025, 6), (5, 4096, 2)])
def test_balance_gradient_of_far_logits(m, T, E, k, zt, shift):
    """The softmax does not depend on where the logits lie, nor does its gradient."""
    z, g = logits(T, E, T * E, "f32")
    z = (z * max(1.0, abs(shift) * 2.0 ** -24) + shift).to(DT[zt])  # at least about one step of fp32 apart
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g).to(torch.int32)
    mask = (torch.rand(T, device="cuda", generator=g) < 0.8).to(torch.uint8)
    for dloss in ((0.7, 0.0), (0.0, 0.2), (-0.4, 0.1)):
        check_balance_grad(z, run_balance(m, z, ids, mask, dloss), dloss, mask)


def test_balance_gradient_of_tokens_left_out_is_0_whatever_the_weights(m):
    z, g = logits(9, 70, 5)
    ids = torch.randint(0, 70, (9, 3), device="cuda", generator=g).to(torch.int32)
    mask = torch.ones(9, dtype=torch.uint8, device="cuda")
    mask[1] = 0
    z[4] = -float("inf")
    for dloss in ((float("inf"), 0.0), (0.0, float("nan"))):
        dz = run_balance(m, z, ids, mask, dloss)["dz"]
        assert torch.all(dz[1] == 0) and torch.all(dz[4] == 0)
        assert torch.isnan(dz[0]).any()


def test_balance_gradient_in_place(m):
    z, g = logits(100, 48, 3)
    ids = z.topk(4, dim=1).indices.to(torch.int32)
    o = run_balance(m, z, ids)
    d = torch.tensor([0.7, 0.2], device="cuda")
    zz = z.clone()
    m.moe_balance_loss_bwd(zz, m.MOE_X_F32, o["lse"].contiguous(), None, o["counts"].contiguous(), o["totals"], d, 100, 48, zz)
    assert torch.equal(zz, o["dz"])


def test_balance_offsets_past_32_bits(m):
    """More than 2^32 logits, all 0 but the last token's."""
    E, T = 512, (1 << 23) + 5
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of device memory")
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    z[T - 1, 3] = 20.0
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[T - 1] = 3
    dev = dict(device="cuda")
    counts, totals = torch.empty(E, dtype=torch.int32, **dev), torch.empty(2, dtype=torch.int32, **dev)
    share, lse, loss = torch.empty(E, dtype=torch.float64, **dev), torch.empty(T, **dev), torch.empty(2, **dev)
    n = m.moe_balance_workspace_bytes(T, E)
    ws = torch.empty(n, dtype=torch.uint8, **dev)
    m.moe_balance_loss(z, m.MOE_X_BF16, ids, None, T, E, 1, counts, totals, share, lse, loss, ws, n)
    d, dz = torch.tensor([0.0, 1.0], **dev), torch.full_like(z, 7.0)
    m.moe_balance_loss_bwd(z, m.MOE_X_BF16, lse, None, counts, totals, d, T, E, dz)
    torch.cuda.synchronize()
    assert counts[0] == T - 1 and counts[3] == 1 and totals.tolist() == [T, T]
    big = np.exp(20.0)
    p3, p = big / (big + E - 1), 1.0 / (big + E - 1)
    want = np.full(E, ((T - 1) / E + p) / T)
    want[3] = ((T - 1) / E + p3) / T
    np.testing.assert_allclose(host64(share), want, rtol=(T + E + 64) * 2.0 ** -52)
    for t, l in ((0, np.log(E)), (T // 2, np.log(E)), (T - 2, np.log(E)), (T - 1, np.log(big + E - 1))):
        assert abs(float(lse[t]) - l) <= 2.0 ** -24 * l * 1.01
        # dz = 2 lse p / n: p of fp32 numbers (an exponent of up to 20 in size, rounded, and lse's rounding: 2^-18
        # relative in all), three products, one rounding to bf16
        q = np.full(E, p if t == T - 1 else 1.0 / E)
        if t == T - 1:
            q[3] = p3
        w = 2 * l * q / T
        assert np.all(np.abs(host64(dz[t]) - w) <= (2.0 ** -8 + 2.0 ** -17) * w)


# ------------------------------------------- together, streams and graphs


def test_decode_head_behind_a_stack(m):
    """Two 4-bit layers, then the head's logits and a draw: each against its reference on what it was given."""
    import synth
    from expert_vram_slot_amd.layer import DecodeHead, SlotStack
    E, k, H, I, S, T, V, group = 16, 4, 256, 128, 16, 5, 3001, 64
    base = synth.config_seed("c4")
    layers = []
    for n in range(2):
        store = synth.slabs(synth.W_Q4B32, base, n, 0, E, H, I, 0.05)
        pinned = torch.empty(store.shape, dtype=torch.uint8, pin_memory=True)
        pinned.copy_(torch.from_numpy(store))
        G = synth.normal(synth.key(base, synth.TAG_G, n, 0), (E, H), 0.5, synth.X_BF16)
        layers.append(dict(host_store=pinned, slot_store=torch.from_numpy(store).cuda(),
                           G=torch.from_numpy(G.view(np.int16)).cuda(),
                           resident=torch.arange(S, dtype=torch.int32, device="cuda")))
    stack = SlotStack(E=E, k=k, H=H, I=I, S=S, w_type=synth.W_Q4B32, T_max=8, layers=layers, n_threads=1)
    g = torch.Generator(device="cuda").manual_seed(6)
    wq, scales, _ = weights(V, H, group, 8)
    head = DecodeHead(H=H, V=V, wq=wq, scales=scales, group=group, T_max=8)
    u, p = torch.rand(T, device="cuda", generator=g), torch.full((T,), 0.9, device="cuda")
    for step in range(3):
        x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
        h = stack.step(x, T, host_pass=False)
        ids, prob = head.step(h, T, u, top_p=p)
        torch.cuda.synchronize()
        want, size = ref.linear_q4(host64(h), wq.cpu().numpy(), scales.cpu().numpy(), group)
        got = host64(head.logits_buf[:T])
        assert np.all(np.abs(got - want) <= (2 * 128 + H / 32 + 8) * 2.0 ** -23 * size)
        for t in range(T):
            i, q, _ = ref.sample_row(got[t], float(u[t]), top_p=float(p[t]))
            assert int(ids[t]) == i and abs(float(prob[t]) - q) <= 2.0 ** -24 * q + V * 2.0 ** -50
        # the last layer's router: profile, gradient, and the bias table its shares make
        L = stack.layer
        b = L.balance(T)
        z, picks = host64(L.logits[:T * E].view(T, E)), L.ids[:T * k].view(T, k).cpu().numpy()
        w = ref.balance(z, picks)
        np.testing.assert_array_equal(b["counts"].cpu().numpy(), w["counts"])
        np.testing.assert_allclose(host64(b["share"]), w["share"], rtol=(T + E + 64) * 2.0 ** -52)
        dz = L.balance_grad(T, torch.tensor([1.0, 0.1], device="cuda"))
        np.testing.assert_allclose(host64(dz), ref.balance_grad(z, picks, np.array([1.0, 0.1])), rtol=1e-4, atol=1e-7)
        bias = torch.empty(E, device="cuda")
        m.moe_bias_table(b["share"], E, 6, -1.0, bias)
        import oracle
        want_bias = oracle.bias_table(host64(b["share"]), 6, -1.0)
        assert np.all(np.abs(bias.cpu().numpy() - want_bias) <= np.spacing(np.abs(want_bias)))


def test_decode_head_takes_x_as_it_lies(m):
    """Rows of a wider matrix, a flat x, one with dimensions between and the bits of bf16 give what a copy gives."""
    from expert_vram_slot_amd.layer import DecodeHead
    H, V, T, group = 256, 1003, 5, 32
    wq, scales, g = weights(V, H, group, 12)
    head = DecodeHead(H=H, V=V, wq=wq, scales=scales, group=group, T_max=8)
    wide = torch.randn(T + 1, 3 * H, device="cuda", generator=g).bfloat16()
    u = torch.rand(T, device="cuda", generator=g)
    k = torch.full((T,), 20, dtype=torch.int32, device="cuda")
    x = wide[:T, H:2 * H].contiguous()
    want = [o.clone() for o in (head.logits(x, T), *head.step(x, T, u, top_k=k))]
    for given in (wide[:, H:2 * H], x.reshape(-1), x.view(T, 1, H), x.view(torch.int16)):
        got = (head.logits(given, T), *head.step(given, T, u, top_k=k))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = head.step(wide[2:3, H:2 * H], 1, u[2:], top_k=k[2:])
    assert all(torch.equal(a, b[2:3]) for a, b in zip(got, want[1:]))
    with pytest.raises(m.MoeError):
        head.logits(torch.zeros(T, H + 4, dtype=torch.bfloat16, device="cuda")[:, :H], T)  # rows 8 bytes off 16
    with pytest.raises(m.MoeError):
        head.logits(x[:1].expand(T, H), T)  # one row for all


def test_layer_balance_of_steps_of_different_sizes(m):
    """The statistics are the last step's, its first tokens' alone too; a graph's step and balance may be of another size."""
    import synth
    from expert_vram_slot_amd.layer import SlotLayer
    E, k, H, I, S = 16, 4, 256, 128, 16
    base = synth.config_seed("c4")
    store = synth.slabs(synth.W_Q4B32, base, 0, 0, E, H, I, 0.05)
    pinned = torch.empty(store.shape, dtype=torch.uint8, pin_memory=True)
    pinned.copy_(torch.from_numpy(store))
    G = synth.normal(synth.key(base, synth.TAG_G, 0, 0), (E, H), 0.5, synth.X_BF16)
    L = SlotLayer(E=E, k=k, H=H, I=I, S=S, w_type=synth.W_Q4B32, T_max=8, policy="static", host_store=pinned,
                  slot_store=torch.from_numpy(store).cuda(), G=torch.from_numpy(G.view(np.int16)).cuda(), n_threads=1)
    L.init_cache(torch.arange(S, dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(8, H, device="cuda", generator=g).bfloat16()
    d = torch.tensor([1.0, 0.1], device="cuda")

    def check(T, mask=None):
        b, dz = L.balance(T, mask), L.balance_grad(T, d, mask)
        z, picks = host64(L.logits[:T * E].view(T, E)), L.ids[:T * k].view(T, k).cpu().numpy()
        mh = None if mask is None else mask[:T].cpu().numpy()
        w = ref.balance(z, picks, mh)
        np.testing.assert_array_equal(b["counts"].cpu().numpy(), w["counts"])
        np.testing.assert_allclose(host64(b["share"]), w["share"], rtol=(T + E + 64) * 2.0 ** -52)
        np.testing.assert_allclose(host64(dz), ref.balance_grad(z, picks, np.array([1.0, 0.1]), mh), rtol=1e-4, atol=1e-7)

    for T in (8, 3):
        L.step(x[:T], T, host_pass=False)
        check(T)
        check(T - 1, torch.arange(8, device="cuda") > 0)  # a mask of bool, longer than the batch
    with pytest.raises(AssertionError):
        L.balance(4)
    L.balance(3)
    L.step(x[:5], 5, host_pass=False)
    with pytest.raises(AssertionError):
        L.balance_grad(3, d)
    check(5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.step(x, 8, host_pass=False)
        L.balance(8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step(x, 8, host_pass=False)
        L.balance(8)
    for rep in range(3):
        L.step(x[:2], 2, host_pass=False)
        check(2)
        x.copy_(torch.randn(8, H, device="cuda", generator=g))
        graph.replay()
        dz = L.balance_grad(8, d).clone()
        check(8)
        assert torch.equal(dz, L.balance_grad(8, d))


def _whole_path(m, T, V, K, group, seed):
    """Buffers and a call of every operator; returns (call, inputs to refill, outputs)."""
    wq, scales, g = weights(V, K, group, seed)
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    y = torch.empty(T, V, device="cuda")
    u = torch.rand(T, device="cuda", generator=g)
    k = torch.full((T,), 60, dtype=torch.int32, device="cuda")
    p = torch.full((T,), 0.9, device="cuda")
    ids, prob = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
    n = m.moe_sample_workspace_bytes(T, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    E, kk = 96, 4
    z = torch.randn(8 * T, E, device="cuda", generator=g)
    picks = z.topk(kk, dim=1).indices.to(torch.int32)
    counts, totals = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    share, lse, loss = torch.empty(E, dtype=torch.float64, device="cuda"), torch.empty(8 * T, device="cuda"), torch.empty(2, device="cuda")
    d, dz = torch.tensor([0.5, 0.1], device="cuda"), torch.empty_like(z)
    bn = m.moe_balance_workspace_bytes(8 * T, E)
    bws = torch.empty(bn, dtype=torch.uint8, device="cuda")

    def call(stream=None):
        m.moe_linear_q4(x, m.MOE_X_BF16, K, wq, scales, group, None, T, V, K, y, m.MOE_X_F32, V, stream)
        m.moe_sample(y, m.MOE_X_F32, V, T, V, None, None, k, p, u, ids, prob, ws, n, stream)
        m.moe_balance_loss(z, m.MOE_X_F32, picks, None, 8 * T, E, kk, counts, totals, share, lse, loss, bws, bn, stream)
        m.moe_balance_loss_bwd(z, m.MOE_X_F32, lse, None, counts, totals, d, 8 * T, E, dz, stream)

    return call, (x, u, z), (y, ids, prob, counts, totals, share, lse, loss, dz)


@pytest.mark.parametrize("T,V", [(1, 5001), (12, 40000), (40, 33000)])
def test_captured_and_replayed_with_eager_calls_between(m, T, V):
    call, inputs, outputs = _whole_path(m, T, V, 512, 32, 1)
    other, _, _ = _whole_path(m, T + 3, V + 77, 256, 64, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(4):
        g = torch.Generator(device="cuda").manual_seed(50 + rep)
        inputs[0].copy_(torch.randn(inputs[0].shape, device="cuda", generator=g))
        inputs[1].copy_(torch.rand(inputs[1].shape, device="cuda", generator=g))
        inputs[2].copy_(torch.randn(inputs[2].shape, device="cuda", generator=g))
        call()
        torch.cuda.synchronize()
        want = [o.clone() for o in outputs]
        for o in outputs:
            o.zero_()
        other()
        graph.replay()
        other()
        torch.cuda.synchronize()
        for a, b in zip(want, outputs):
            assert torch.equal(a, b)


def test_two_streams_with_workspaces_of_their_own(m):
    paths = [_whole_path(m, T, 33000, 512, 32, T) for T in (6, 40)]
    want = []
    for call, _, outputs in paths:
        call()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outputs])
        for o in outputs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in paths]
    for rep in range(5):
        for (call, _, _), s in zip(paths, streams):
            call(s)
    torch.cuda.synchronize()
    for (_, _, outputs), w in zip(paths, want):
        for a, b in zip(w, outputs):
            assert torch.equal(a, b)
