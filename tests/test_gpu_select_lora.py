"""moe_route_select, moe_bias_balance and moe_lora_add against plain references in 64 bits.

Tolerances:
  select ids        equal: choices are compared as doubles, and random ones are never as close as a double's rounding
  select w          one rounding to fp32 (2^-24) of a double, for renormalised weights and sigmoids; a raw softmax may
                    divide by a sum of E exponentials in fp32: each of them is off by (1.5 |z - m| + 2) * 2^-23 (the
                    argument's rounding twice over, the exponential's last bit), in the mean over p at most
                    (1.5 ln E + 2) * 2^-23 (sum p |z - m| <= ln E: the softmax's entropy is at most ln E, and lse >= m),
                    and E / 64 + 6 additions follow: (E / 64 + 1.5 ln E + 8) * 2^-23 is DS(E) below; the pick's own
                    exponential besides
  select dz         fp32 of terms good to the above: 3 * DS(E) of the magnitudes that are added up (p twice, the sum over
                    the picks), one rounding each of the part, of dz_add + part and of the output's type
  lora, exact       bits: whole numbers and powers of two, every partial sum a whole number below 2^24
  lora, random      each output passes K + r + 8 roundings at most, of 2^-23 (a matrix instruction may cut off) of a
                    partial sum below the sum of the magnitudes; bf16 outputs add half a step, 2^-8 of the value
"""
import numpy as np
import pytest

import select_lora_reference as ref

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
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def code(m, name):
    return m.MOE_X_BF16 if name == "bf16" else m.MOE_X_F32


def name_of(t):
    return "bf16" if t.dtype == torch.bfloat16 else "f32"


def host64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ select


def DS(E):
    return (E / 64 + 1.5 * np.log(E) + 8) * 2.0 ** -23


def run_select(m, z, k, rule, bias=None, mask=None, ids_in=None):
    T, E = z.shape
    ids = torch.full((T + 1, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -9.0, device="cuda")
    m.moe_route_select(z, code(m, name_of(z)), bias, mask, ids_in, T, E, k, m.select_rule(**rule), ids, w)
    torch.cuda.synchronize()
    assert torch.all(ids[T] == -9) and torch.all(w[T] == -9.0)
    return ids[:T], w[:T]


def plain(rule):
    """A rule as the reference takes it."""
    a = dict(score="softmax", groups=1, groups_kept=None, group_top=1, renorm=True, scale=1.0)
    a.update(rule)
    return dict(score=a["score"], groups=a["groups"], kept=a["groups_kept"] or a["groups"], top=a["group_top"],
                renorm=a["renorm"], scale=a["scale"])


def w_bound(z, ids, want, r, E):
    """How far w may be off."""
    tol = 2.0 ** -24 + 2.0 ** -45
    if r["score"] == "softmax" and not r["renorm"]:
        zz = np.where(z > -np.inf, z, -np.inf)
        with np.errstate(invalid="ignore"):
            d = np.nan_to_num(zz.max(axis=1, keepdims=True) - np.take_along_axis(zz, np.clip(ids, 0, E - 1), axis=1),
                              nan=0.0, posinf=0.0)
        tol = tol + DS(E) + (1.5 * np.minimum(d, 200) + 4) * 2.0 ** -23
    return tol * np.abs(want) + 1.2e-38  # below the normal range: as good as 0


def check_select(m, z, k, rule, bias=None, mask=None, ids_in=None):
    ids, w = run_select(m, z, k, rule, bias, mask, ids_in)
    zh, r = host64(z), plain(rule)
    want_ids, want, _ = ref.select(zh, k, bias=None if bias is None else host64(bias),
                                   mask=None if mask is None else mask.cpu().numpy(),
                                   ids_in=None if ids_in is None else ids_in.cpu().numpy(), **r)
    if ids_in is None:
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    else:
        assert torch.all(ids == -9)  # not written
    got = host64(w)
    assert np.all(np.abs(got - want) <= w_bound(zh, want_ids, want, r, z.shape[1])), np.abs(got - want).max()
    return ids, w


def check_grad(m, z, ids, dw, rule, add=None, into=None):
    T, E = z.shape
    k, r, zt = ids.shape[1], plain(rule), name_of(z)
    zh, ih, ah = host64(z), ids.cpu().numpy(), 0.0 if add is None else host64(add)
    if into is None:
        into = torch.full((T * E + 1,), 5.0, dtype=z.dtype, device="cuda")
    m.moe_route_select_bwd(z, code(m, zt), ids, dw, T, E, k, m.select_rule(**rule), add, into)
    torch.cuda.synchronize()
    got = host64(into.reshape(-1)[:T * E].view(T, E))
    if into.numel() > T * E:
        assert float(into[T * E]) == 5.0
    part, size = ref.select_grad(zh, ih, host64(dw), r["score"], r["renorm"], r["scale"])
    want = part + ah
    with np.errstate(invalid="ignore"):
        top = np.where(np.isfinite(zh), zh, -np.inf).max(axis=1, keepdims=True)
        far = np.abs(np.nan_to_num(np.where(np.isfinite(zh), zh - top, 0)))
    own = (1.5 * np.minimum(far, 200) + 4) * 2.0 ** -23 if r["score"] == "softmax" and not r["renorm"] else 0.0
    # numbers below 2^-126 = 1.1755e-38 are as good as 0: one of dz, and one of p, which goes into dz times h - sum h p, of a
    # magnitude of 2 max |h| at most (sum p <= 1): off by 2^-126 (1 + 2 max |h|) together
    h = r["scale"] * np.abs(np.nan_to_num(np.where(ih >= 0, host64(dw), 0))).max(axis=1, keepdims=True)
    tol = (3 * DS(E) + own) * size + 2.0 ** -23 * (np.abs(ah) + np.abs(part)) + HALF[zt] * np.abs(want) * (1 + 2.0 ** -8) + 1.2e-38 * (1 + 2 * h)
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) - tol).max()
    return into


def logits(T, E, seed, zt="f32", scale=1.5):
    g = gen(seed)
    return (scale * torch.randn(T, E, device="cuda", generator=g)).to(DT[zt])


RULES = [dict(score="softmax"), dict(score="softmax", renorm=False, scale=2.5), dict(score="sigmoid", scale=2.5),
         dict(score="sigmoid", renorm=False)]
SHAPES = [  # T, E, k, groups, kept, top
    (1, 1, 1, 1, 1, 1), (1, 8, 2, 1, 1, 1), (3, 5, 5, 1, 1, 1), (7, 64, 8, 8, 3, 2), (16, 65, 6, 5, 2, 1), (33, 127, 3, 1, 1, 1),
    (64, 128, 8, 1, 1, 1), (9, 128, 32, 2, 1, 2), (17, 129, 4, 3, 2, 2), (65, 288, 8, 8, 4, 2), (33, 288, 8, 1, 1, 1),
    (12, 320, 10, 64, 9, 1), (12, 512, 10, 16, 3, 2), (40, 513, 32, 27, 20, 2), (8, 1024, 16, 1, 1, 1),
    (5, 1025, 7, 41, 5, 2), (3, 2048, 12, 32, 4, 1), (4, 4096, 32, 64, 64, 2), (2, 4095, 8, 1, 1, 1), (130, 16, 4, 16, 5, 2),
    (257, 96, 6, 3, 1, 2)]


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
@pytest.mark.parametrize("T,E,k,groups,kept,top", SHAPES)
def test_select_matches_reference(m, T, E, k, groups, kept, top, rule, with_bias, zt):
    rule = dict(rule, groups=groups, groups_kept=kept, group_top=top)
    z = logits(T, E, T * E + k, zt)
    g = gen(E)
    bias = 0.001 * torch.randint(-80, 81, (E,), device="cuda", generator=g).float() if with_bias else None
    mask = (torch.rand(T, device="cuda", generator=g) < 0.8).to(torch.uint8) if T > 30 else None
    ids, _ = check_select(m, z, k, rule, bias, mask)
    dw = torch.randn(T, k, device="cuda", generator=g)
    check_grad(m, z, ids, dw, rule)
    check_grad(m, z, ids, dw, rule, add=logits(T, E, 9, zt, 0.1))


@pytest.mark.parametrize("levels", [1, 2, 5, 40])
@pytest.mark.parametrize("E,k,groups,kept", [(7, 3, 1, 1), (64, 8, 4, 2), (288, 8, 8, 4), (300, 32, 1, 1), (1000, 10, 1, 1),
                                             (2048, 20, 16, 3)])
def test_select_ties(m, E, k, groups, kept, levels):
    """Logits and biases of a few values each: the border lies among equals, and ids decide."""
    g = gen(E + levels)
    z = torch.randint(0, levels, (24, E), device="cuda", generator=g).float() * 0.5 - 0.25
    z[1] = torch.where(z[1] == -0.25, torch.zeros_like(z[1]), z[1])
    z[1, ::2] = torch.where(z[1, ::2] == 0, -torch.zeros_like(z[1, ::2]), z[1, ::2])  # -0 and 0 are equal
    z[2] = 90.0 + z[2]    # sigmoids of 1 all
    z[3] = -900.0 + z[3]  # and of 0
    for score, top in (("sigmoid", 1), ("softmax", 2)):
        rule = dict(score=score, groups=groups, groups_kept=kept, group_top=top)
        check_select(m, z, k, rule)
        check_select(m, z, k, rule, torch.zeros(E, device="cuda"))
        check_select(m, z, k, rule, torch.randint(0, 2, (E,), device="cuda", generator=g).float() * 0.25)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(64, 6), (288, 8), (1500, 12)])
def test_select_choices_closer_than_fp32(m, E, k, score):
    """Biases make up for the logits but for some 1e-10: only 64-bit scores tell the experts apart."""
    g = gen(E)
    z = torch.randn(16, E, device="cuda", generator=g)
    one = z[:1].expand(16, E).contiguous()  # the same token over and over: its scores and a constant make the bias
    s = ref.scores(host64(one), score)[0]
    bias = torch.from_numpy((0.75 - s).astype(np.float32)).cuda()
    c = s + host64(bias)
    assert len(np.unique(c.astype(np.float32))) < E / 8 and len(np.unique(c)) == E
    check_select(m, one, k, dict(score=score), bias)
    check_select(m, one, k, dict(score=score, groups=4, groups_kept=2, group_top=2), bias)
    check_select(m, z, k, dict(score=score), bias)


@pytest.mark.parametrize("shift", [0.0, 3.0, -20.0, 300.0])
@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(64, 6, 1), (288, 8, 1), (512, 10, 1), (1500, 12, 1), (288, 8, 8)])
def test_select_pairs_closer_than_fp32(m, E, k, groups, score, zt, shift):
    """Of every two of the best, the second's bias makes up for its logit but for some 1e-9; the others lie far off."""
    g = gen(E + k)
    z = logits(1, E, E, zt).expand(24, E).contiguous()
    z = (z.float() + (shift if score == "softmax" else 0.0)).to(DT[zt])
    z[20:] = logits(4, E, E + 1, zt)  # and tokens that the biases are not made for
    s = ref.scores(host64(z[:1]), score)[0]
    order = np.argsort(-s, kind="stable")
    bias = np.zeros(E, np.float32)
    for i in range(0, 2 * (k // 2) + 2, 2):
        bias[order[i + 1]] = np.float32(s[order[i]] - s[order[i + 1]])
    bias = torch.from_numpy(bias).cuda()
    check_select(m, z, k, dict(score=score, groups=groups, groups_kept=max(1, groups // 2), group_top=2), bias)
    check_select(m, z, k, dict(score=score, groups=groups, groups_kept=max(1, groups // 2), renorm=False), bias)


def special_rows(E, g):
    inf, nan = float("inf"), float("nan")
    z = torch.randn(12, E, device="cuda", generator=g)
    z[0] = -inf                                     # nothing left
    z[1] = nan
    z[2], z[2, E - 1] = -inf, -3e38                 # one expert, near the type's lowest value
    z[3, ::2] = -inf
    z[4, ::2] = nan
    z[5, 1], z[5, E // 2] = inf, inf                # two outweigh the rest
    z[6] = torch.finfo(torch.float32).min           # a mask of the lowest value, everywhere
    z[7], z[7, E // 3] = torch.finfo(torch.float32).min, 1.0
    z[8] = torch.where(torch.rand(E, device="cuda", generator=g) < 0.5, 1e-45, -1e-45)  # below the normal range
    z[9] = 3e38
    z[10] = 200.0 * z[10]
    z[11] = inf
    return z


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
@pytest.mark.parametrize("E,k,groups,kept", [(6, 3, 1, 1), (96, 8, 8, 4), (288, 32, 1, 1), (2048, 8, 32, 3)])
def test_select_masked_and_special_rows(m, E, k, groups, kept, rule):
    g = gen(E)
    rule = dict(rule, groups=groups, groups_kept=kept, group_top=2)
    for zt in ("f32", "bf16"):
        z = special_rows(E, g).to(DT[zt])
        ids, _ = check_select(m, z, k, rule)
        dw = torch.randn(12, k, device="cuda", generator=g)
        check_grad(m, z, ids, dw, rule)
        dead = torch.where(ids < 0, torch.full_like(dw, float("nan")), dw)  # what belongs to no pick is not used
        check_grad(m, z, ids, dead, rule)
        bias = torch.randn(E, device="cuda", generator=g)
        bias[::3], bias[1] = -float("inf"), float("nan")
        check_select(m, z, k, rule, bias)
        mask = torch.tensor([1, 0, 1, 1, 0, 1, 0, 1, 1, 2, 1, 0], dtype=torch.uint8, device="cuda")
        check_select(m, z, k, rule, bias, mask)
        check_select(m, z, k, rule, torch.full((E,), -float("inf"), device="cuda"))  # no expert open at all


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
@pytest.mark.parametrize("E,k,groups", [(64, 6, 1), (300, 8, 1), (512, 10, 1), (512, 4, 8), (1024, 32, 1), (4096, 8, 1)])
def test_select_signalling_nans(m, E, k, groups, rule):
    """Neither an expert whose logit is a signalling NaN nor one that is looked at next to it is lost or found by that."""
    z = logits(70, E, 17 * E + k)
    z[20:40] = 8.0 * z[20:40] + 20.0
    z[40:50] = torch.floor(z[40:50])
    g = gen(5)
    holes = torch.rand(70, E, device="cuda", generator=g) < 0.4
    holes[:10], holes[10:20] = False, False
    holes[:60, E - E // 8:] |= True  # the last that each lane holds
    rule = dict(rule, groups=groups, group_top=2)
    for zt, bits, ints in (("f32", 0x7F800001, torch.int32), ("bf16", 0x7F81, torch.int16)):
        zz = z.to(DT[zt]).clone()
        zz.view(ints)[holes] = bits
        assert torch.equal(torch.isnan(zz), holes)
        ids, _ = check_select(m, zz, k, rule)
        check_grad(m, zz, ids, torch.randn(70, k, device="cuda", generator=g), rule)
        check_select(m, zz, k, rule, torch.randn(E, device="cuda", generator=g))


def test_select_biases_without_end(m):
    """+inf picks an expert whatever its score; the type's largest values stay finite in double."""
    z = logits(20, 64, 3)
    bias = torch.zeros(64, device="cuda")
    bias[7], bias[41], bias[3], bias[50] = float("inf"), float("inf"), 3.4e38, -3.4e38
    for rule in (dict(score="sigmoid"), dict(score="softmax", groups=8, groups_kept=3, group_top=2)):
        ids, _ = check_select(m, z, 5, rule, bias)
        assert torch.all((ids[:, 0] == 7) | (ids[:, 0] == 41))


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
@pytest.mark.parametrize("E", [5, 200, 1100])
def test_select_of_given_picks(m, E, rule):
    """Given picks, out of range and repeated ones among them: weights and gradients."""
    T, k = 37, 4
    g = gen(E)
    z = logits(T, E, E)
    z[3, :] = -float("inf")
    z[4, 0], z[5, 1] = float("nan"), -float("inf")
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g).to(torch.int32)
    ids[0, 1], ids[1, 0], ids[2], ids[4, 0], ids[5, 1] = -1, E, -1, 0, 1
    ids[6] = 2
    ids[7, 0] = ids[7, 3]
    ids[8, 0], ids[8, 1] = 2 ** 31 - 1, -2 ** 31
    check_select(m, z, k, rule, ids_in=ids)
    dw = torch.randn(T, k, device="cuda", generator=g)
    check_grad(m, z, ids, dw, rule)
    mask = (torch.arange(T, device="cuda") % 3 > 0).to(torch.uint8)
    _, w = check_select(m, z, k, rule, ids_in=torch.where(mask[:, None] > 0, ids, -1))
    assert torch.equal(w, run_select(m, z, k, rule, None, mask, ids)[1])


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
def test_select_gradient_against_differences(m, rule):
    """The gradient of the kernel's own weights: central differences of a step of 2^-6 in z, at the picks that the
    unmoved logits take."""
    T, E, k = 4, 24, 5
    z = logits(T, E, 21, scale=1.0)
    ids, _ = run_select(m, z, k, rule)
    dw = torch.randn(T, k, device="cuda", generator=gen(1))
    dz = host64(check_grad(m, z, ids, dw, rule)[:T * E].view(T, E))
    h, d64 = 2.0 ** -6, host64(dw)
    for e in range(E):
        f = []
        for s in (h, -h):
            zz = z.clone()
            zz[:, e] += s
            f.append((host64(run_select(m, zz, k, rule, ids_in=ids)[1]) * d64).sum(axis=1))
        # truncation h^2 / 6 times a third derivative below scale * sum |dw| (each weight's is below 1), rounding of w,
        # (2^-24 + DS) twice over 2 h
        scale = plain(rule)["scale"] * np.abs(d64).sum(axis=1)
        assert np.all(np.abs(dz[:, e] - (f[0] - f[1]) / (2 * h)) <= scale * (h * h / 6 + (2.0 ** -23 + 2 * DS(E) + 2.0 ** -19) / h))


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
@pytest.mark.parametrize("zt", ["f32", "bf16"])
def test_select_gradient_in_place(m, rule, zt):
    T, E, k = 70, 130, 6
    z, add = logits(T, E, 5, zt), logits(T, E, 6, zt, 0.1)
    ids, _ = run_select(m, z, k, rule)
    dw = torch.randn(T, k, device="cuda", generator=gen(2))
    want = check_grad(m, z, ids, dw, rule, add)[:T * E].view(T, E)
    for into_z in (True, False):
        z2, add2 = z.clone(), add.clone()
        into = z2 if into_z else add2
        m.moe_route_select_bwd(z2, code(m, zt), ids, dw, T, E, k, m.select_rule(**rule), add2, into)
        assert torch.equal(into, want)


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
def test_select_of_far_logits(m, rule):
    """Softmaxes do not see where the logits lie; sigmoids far out are renormalised by ratios."""
    for shift in (1e4, -1e4, 90.0, -90.0):
        z = logits(33, 100, 8) + shift
        ids, _ = check_select(m, z, 6, rule)
        check_grad(m, z, ids, torch.randn(33, 6, device="cuda", generator=gen(3)), rule)


@pytest.mark.parametrize("T", [4000, 70001])
def test_select_many_tokens(m, T):
    """Whole batches against a batch of one token at a time's worth of reference: every 97th token, and all of them
    against the same tokens in another order."""
    E, k = 288, 8
    z = logits(T, E, T)
    bias = 0.001 * torch.randint(-60, 61, (E,), device="cuda", generator=gen(1)).float()
    rule = dict(score="sigmoid", groups=8, groups_kept=4, group_top=2, scale=2.5)
    ids, w = run_select(m, z, k, rule, bias)
    some = torch.arange(0, T, 97, device="cuda")
    some_ids, some_w = check_select(m, z[some].contiguous(), k, rule, bias)
    assert torch.equal(ids[some], some_ids) and torch.equal(w[some], some_w)
    back = torch.arange(T - 1, -1, -1, device="cuda")
    i2, w2 = run_select(m, z[back].contiguous(), k, rule, bias)
    assert torch.equal(ids[back], i2) and torch.equal(w[back], w2)


def test_select_offsets_past_32_bits(m):
    """Logits past 4 GiB: the last tokens' picks and gradient."""
    T, E, k = (1 << 21) + 700, 520, 4
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB of device memory")
    z = torch.zeros(T, E, device="cuda")
    tail = logits(700, E, 4)
    z[-700:] = tail
    rule = dict(score="softmax", renorm=False)
    ids, w = run_select(m, z, k, rule)
    some_ids, some_w = check_select(m, tail, k, rule)
    assert torch.equal(ids[-700:], some_ids) and torch.equal(w[-700:], some_w)
    assert torch.all(ids[:-700] == torch.arange(k, device="cuda"))
    dw = torch.zeros(T, k, device="cuda")
    dw[-700:] = torch.randn(700, k, device="cuda", generator=gen(8))
    m.moe_route_select_bwd(z, m.MOE_X_F32, ids, dw, T, E, k, m.select_rule(**rule), None, z)
    want = check_grad(m, tail, some_ids, dw[-700:].contiguous(), rule)[:700 * E].view(700, E)
    assert torch.equal(z[-700:], want) and not torch.any(z[:-700])


# ------------------------------------------------------------ logits, bias


@pytest.mark.parametrize("T,H,E", [(1, 64, 8), (3, 256, 17), (40, 2048, 128), (600, 512, 96), (520, 264, 33)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_route_logits_are_moe_routes(m, T, H, E, xt):
    g = gen(T + H)
    x, G = torch.randn(T, H, device="cuda", generator=g).to(DT[xt]), torch.randn(E, H, device="cuda", generator=g).to(DT[xt])
    a, b = torch.full((T * E + 1,), 5.0, device="cuda"), torch.empty(T, E, device="cuda")
    ids, w = torch.empty(T, 1, dtype=torch.int32, device="cuda"), torch.empty(T, 1, device="cuda")
    m.moe_route_logits(x, code(m, xt), G, T, H, E, a)
    m.moe_route(x, code(m, xt), G, None, None, T, H, E, 1, ids, w, b)
    assert torch.equal(a[:T * E].view(T, E), b) and float(a[-1]) == 5.0
    # doubles summed and rounded once
    want = host64(x) @ host64(G).T
    size = np.abs(host64(x)) @ np.abs(host64(G)).T
    assert np.all(np.abs(host64(b) - want) <= 2.0 ** -24 * np.abs(want) + (H + 8) * 2.0 ** -53 * size)


@pytest.mark.parametrize("L,E", [(1, 1), (1, 288), (3, 7), (48, 512), (5, 4096), (700, 65)])
def test_bias_balance(m, L, E):
    g = gen(L * E)
    counts = torch.randint(0, 6 if E % 2 else 3000, (L, E), device="cuda", generator=g).to(torch.int32)
    bias = 0.001 * torch.randint(-60, 61, (L, E), device="cuda", generator=g).float()
    bias[torch.rand(L, E, device="cuda", generator=g) < 0.1] = -float("inf")
    bias[0, 0] = float("nan")
    if L > 1:
        counts[1] = 5            # even: nothing moves
        bias[L - 1] = -float("inf")  # no expert open
    if E > 5:
        counts[0, 3], counts[0, 4] = 2 ** 31 - 1, 2 ** 31 - 2
        bias[0, 5] = float("inf")
    out = torch.full((L * E + 1,), 5.0, device="cuda")
    m.moe_bias_balance(counts, bias, L, E, 0.003, out)
    want = ref.bias_balance(counts.cpu().numpy(), bias.cpu().numpy(), 0.003)
    np.testing.assert_array_equal(out[:-1].view(L, E).cpu().numpy(), want)
    assert float(out[-1]) == 5.0
    m.moe_bias_balance(counts, bias, L, E, 0.003, bias)  # in place
    np.testing.assert_array_equal(bias.cpu().numpy(), want)


# -------------------------------------------------------------------- lora


def run_lora(m, x, a, b, ids, ranks=None, scale=None, base=None, yt="f32", pad=(0, 0, 0), in_place=False, stream=None):
    """moe_lora_add on padded copies; the padding of y must stay as it was."""
    (T, K), (n, r, _), N = x.shape, a.shape, b.shape[1]
    ldx, ldb, ldy = K + pad[0], N + pad[1], N + pad[2]
    xp = torch.full((T, ldx), float("nan"), dtype=x.dtype, device="cuda")
    xp[:, :K] = x
    y = torch.full((T + 1, ldy), 77.0, dtype=DT[yt], device="cuda")
    bp = None
    if in_place:
        ldb = ldy
        y[:T, :N] = base
        bp = y
    elif base is not None:
        bp = torch.full((T, ldb), float("nan"), dtype=DT[yt], device="cuda")
        bp[:, :N] = base
    size = m.moe_lora_workspace_bytes(T, K, r)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")  # NaN: needs no clearing
    m.moe_lora_add(xp, code(m, name_of(x)), ldx, a, b, ranks, scale, ids, n, r, T, N, K, bp, ldb, y, code(m, yt), ldy, ws,
                   size, stream)
    torch.cuda.synchronize()
    assert torch.all(y[T] == 77.0) and torch.all(y[:, N:] == 77.0) and torch.all(ws[size:] == 255)
    return y[:T, :N]


def pool(n, r, K, N, g, whole=False):
    if whole:
        a = torch.randint(-2, 3, (n, r, K), device="cuda", generator=g)
        b = torch.randint(-2, 3, (n, N, r), device="cuda", generator=g)
    else:
        a, b = torch.randn(n, r, K, device="cuda", generator=g) * K ** -0.5, torch.randn(n, N, r, device="cuda", generator=g)
    return a.bfloat16(), b.bfloat16()


def some_ids(T, n, kind, g):
    if kind == "runs":
        return (torch.arange(T, device="cuda") * n // T).to(torch.int32)
    ids = torch.randint(-1, n + 1, (T,), device="cuda", generator=g).to(torch.int32)  # -1 and n: none
    if kind == "one":
        ids = torch.full_like(ids, n - 1)
    return ids


LORA = [  # T, N, K, n, r
    (1, 1, 8, 1, 8), (1, 17, 64, 3, 16), (2, 100, 136, 2, 8), (3, 64, 256, 5, 24), (7, 501, 1536, 5, 24), (15, 33, 40, 4, 32),
    (16, 256, 512, 16, 16), (17, 300, 520, 3, 40), (31, 130, 1000, 40, 64), (33, 1000, 264, 7, 8), (64, 2049, 512, 16, 16),
    (65, 31, 2048, 9, 128), (100, 257, 96, 100, 16), (129, 640, 384, 4, 256), (257, 777, 512, 64, 32), (300, 48, 4096, 2, 56),
    (1000, 129, 72, 8, 64), (2049, 300, 256, 8, 16), (1, 5000, 4096, 2, 16), (4, 40000, 256, 4, 8)]


@pytest.mark.parametrize("kind", ["mixed", "runs", "one"])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K,n,r", LORA)
def test_lora_exact(m, T, N, K, n, r, xt, kind):
    # |h| <= 4 K at most; 2 r |h| + |base|, times a scale of up to 4: in all below 2^24 for typical signs, and checked
    g = gen(T + N + K)
    a, b = pool(n, r, K, N, g, whole=True)
    x = torch.randint(-2, 3, (T, K), device="cuda", generator=g).to(DT[xt])
    ids = some_ids(T, n, kind, g)
    ranks = torch.randint(-1, r + 3, (n,), device="cuda", generator=g).to(torch.int32) if T % 2 else None
    scale = torch.pow(2.0, torch.randint(-1, 3, (n,), device="cuda", generator=g).float()) if N % 2 else None
    base = torch.randint(-64, 65, (T, N), device="cuda", generator=g).float()
    want, size = ref.lora(host64(x), host64(a), host64(b), ids.cpu().numpy(), None if ranks is None else ranks.cpu().numpy(),
                          None if scale is None else host64(scale), host64(base))
    exact = size < 2 ** 22  # in units of a half every partial sum of any order stays below 2^23
    got = host64(run_lora(m, x, a, b, ids, ranks, scale, base, pad=(8, 3, 1)))
    np.testing.assert_array_equal(got[exact], want[exact])
    assert np.all(np.abs(got - want) <= (K + r + 8) * 2.0 ** -23 * size)
    assert np.array_equal(got, host64(run_lora(m, x, a, b, ids, ranks, scale, base, in_place=True, pad=(16, 0, 5))))
    rounded = host64(torch.from_numpy(want).float().to(torch.bfloat16))
    got = host64(run_lora(m, x, a, b, ids, ranks, scale, base.bfloat16(), yt="bf16", pad=(0, 1, 3)))
    np.testing.assert_array_equal(got[exact], rounded[exact])


@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,N,K,n,r", LORA)
def test_lora_random(m, T, N, K, n, r, xt, yt, kind):
    g = gen(T * N + K)
    a, b = pool(n, r, K, N, g)
    x = torch.randn(T, K, device="cuda", generator=g).to(DT[xt])
    ids = some_ids(T, n, kind, g)
    ranks = torch.randint(1, r + 1, (n,), device="cuda", generator=g).to(torch.int32) if K % 3 else None
    scale = 0.5 + torch.rand(n, device="cuda", generator=g)
    base = torch.randn(T, N, device="cuda", generator=g).to(DT[yt]) if T % 3 else None
    want, size = ref.lora(host64(x), host64(a), host64(b), ids.cpu().numpy(), None if ranks is None else ranks.cpu().numpy(),
                          host64(scale), None if base is None else host64(base))
    got = host64(run_lora(m, x, a, b, ids, ranks, scale, base, yt))
    tol = (K + r + 8) * 2.0 ** -23 * size + (2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) if yt == "bf16" else 0)
    assert np.all(np.abs(got - want) <= tol)
    # over all outputs the roundings' signs are as good as random, and a partial sum of K terms is about sqrt(K) of them:
    # sqrt(K) + sqrt(3 r) + 4 times 2^-23 of the outputs' size (an A x kept in bf16 would be off by 2^-9)
    if yt == "f32" and want.size >= 1000:
        assert np.linalg.norm(got - want) <= (np.sqrt(K) + np.sqrt(3 * r) + 4) * 2.0 ** -23 * np.linalg.norm(want)


@pytest.mark.parametrize("kind", ["mixed", "runs", "one"])
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,N,K,n,r", [(1025, 130, 136, 3, 40), (1100, 70, 264, 5, 72), (1500, 200, 96, 2, 128), (2100, 67, 72, 9, 256),
                                       (1030, 1, 8, 2, 136), (1200, 64, 256, 1200, 8), (1090, 129, 512, 70, 64)])
def test_lora_many_tokens_of_large_ranks(m, T, N, K, n, r, xt, yt, kind):
    """Tiles of 64 tokens at every size of h, whole and in part, adapters of every rank."""
    g = gen(T + r)
    a, b = pool(n, r, K, N, g, whole=True)
    x = torch.randint(-2, 3, (T, K), device="cuda", generator=g).to(DT[xt])
    ids = some_ids(T, n, kind, g)
    ranks = torch.randint(0, r + 1, (n,), device="cuda", generator=g).to(torch.int32) if T % 4 else None
    base = torch.randint(-64, 65, (T, N), device="cuda", generator=g).float()
    args = (host64(x), host64(a), host64(b), ids.cpu().numpy(), None if ranks is None else ranks.cpu().numpy())
    for given in (base, None):
        want, size = ref.lora(*args, None, None if given is None else host64(given))
        exact = size < 2 ** 23
        assert exact.mean() > 0.5
        got = host64(run_lora(m, x, a, b, ids, ranks, None, given, "f32", pad=(8, 1, 2)))
        np.testing.assert_array_equal(got[exact], want[exact])
        if given is not None:
            got = host64(run_lora(m, x, a, b, ids, ranks, None, given.to(DT[yt]), yt, in_place=True))
            np.testing.assert_array_equal(got[exact], host64(torch.from_numpy(want).float().to(DT[yt]))[exact])


def test_lora_leaves_the_base_of_others_as_it_is(m):
    """Without an adapter y is base bit for bit: negative zeros, infinities, numbers below the normal range."""
    for yt, T in (("f32", 5), ("bf16", 70), ("f32", 1200)):
        a, b = pool(2, 16, 64, 200, gen(1))
        base = torch.randn(T, 200, device="cuda", generator=gen(2)).to(DT[yt])
        base[:, ::5], base[:, 1::5], base[:, 2::7] = -0.0, float("inf"), 1e-40
        ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        ids[::3] = 1
        ranks = torch.tensor([16, 0], dtype=torch.int32, device="cuda")
        got = run_lora(m, torch.randn(T, 64, device="cuda").bfloat16(), a, b, ids, ranks, None, base, yt)
        kind = torch.int32 if yt == "f32" else torch.int16
        assert torch.equal(got.contiguous().view(kind), base.view(kind))


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_lora_every_weight_by_itself(m, xt):
    """One input of a token, one row of A and one column of B: the product of three, with all 24 bits of an fp32 x."""
    T, N, K, n, r = 48, 70, 264, 3, 24
    g = gen(5)
    bits = 24 if xt == "f32" else 8
    v = torch.randint(1 << (bits - 1), 1 << bits, (T,), device="cuda", generator=g).float()
    ids = (torch.arange(T, device="cuda") % n).to(torch.int32)
    for k0 in range(0, K, 40):
        a, b = torch.zeros(n, r, K, device="cuda"), torch.zeros(n, N, r, device="cuda")
        x = torch.zeros(T, K, device="cuda")
        at = (k0 + torch.arange(T, device="cuda") * 5) % K
        x[torch.arange(T, device="cuda"), at] = v
        for i in range(n):
            j = (k0 // 8 + 5 * i) % r
            a[i, j] = torch.pow(2.0, (torch.arange(K, device="cuda") % 7 - 3).float())
            b[i, :, j] = torch.pow(2.0, (torch.arange(N, device="cuda") % 5 - 2).float())
        got = run_lora(m, x.to(DT[xt]), a.bfloat16(), b.bfloat16(), ids)
        p = torch.pow(2.0, (at % 7 - 3).float())[:, None] * torch.pow(2.0, (torch.arange(N, device="cuda") % 5 - 2).float())
        assert torch.equal(got, v[:, None] * p)


@pytest.mark.parametrize("T,N,K,n,r", [(5, 100, 256, 3, 16), (40, 600, 512, 6, 32), (300, 200, 256, 4, 16), (2100, 260, 128, 4, 64)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_lora_keeps_tokens_and_adapters_apart(m, T, N, K, n, r, xt):
    """Infinities and NaN of a token or an adapter stay there; what lies behind a rank does not matter; a token's bits do
    not depend on its place."""
    g = gen(T)
    a, b = pool(n, r, K, N, g)
    x = torch.randn(T, K, device="cuda", generator=g).to(DT[xt])
    ids = (torch.arange(T, device="cuda") % (n + 1) - 1).to(torch.int32)  # -1: none
    ranks = torch.tensor([r - 3, 0, r // 2 + 1][:n] + [r] * (n - 3), dtype=torch.int32, device="cuda")
    base = torch.randn(T, N, device="cuda", generator=g)
    want = run_lora(m, x, a, b, ids, ranks, None, base)
    assert torch.equal(want[ids < 0], base[ids < 0]) and torch.equal(want[ids == 1], base[ids == 1])
    a2, b2, x2 = a.clone(), b.clone(), x.clone()
    for i in range(n):
        a2[i, int(ranks[i]):] = float("nan")
        b2[i, :, int(ranks[i]):] = float("inf")
    assert torch.equal(run_lora(m, x, a2, b2, ids, ranks, None, base), want)
    x2[T - 1], x2[1] = float("nan"), float("inf")
    x2[0] = float("nan")  # has no adapter
    a2[2] = float("nan")
    got = run_lora(m, x2, a2, b2, ids, ranks, None, base)
    bad = (ids == 2) | (torch.arange(T, device="cuda") == T - 1) | (torch.arange(T, device="cuda") == 1)
    bad &= (ids >= 0) & (ids != 1)
    assert torch.equal(got[~bad], want[~bad]) and not torch.any(torch.isfinite(got[bad]))
    b2[0], scale = float("inf"), torch.ones(n, device="cuda")
    scale[1] = float("nan")  # of an adapter of rank 0
    got = run_lora(m, x, a, b2, ids, ranks, scale, base)
    assert torch.equal(got[ids != 0], want[ids != 0]) and not torch.any(torch.isfinite(got[ids == 0]))
    back = torch.arange(T - 1, -1, -1, device="cuda")
    assert torch.equal(run_lora(m, x[back], a, b, ids[back].contiguous(), ranks, None, base[back]), want[back])


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40])
def test_lora_scales_with_its_input(m, T, xt):
    """Powers of two go through every rounding, in all 24 bits of A x."""
    g = gen(T)
    a, b = pool(3, 16, 512, 300, g)
    x = torch.randn(T, 512, device="cuda", generator=g)
    x = torch.where(x.abs() < 2.0 ** -10, torch.ones_like(x), x).to(DT[xt])
    ids = (torch.arange(T, device="cuda") % 3).to(torch.int32)
    want = run_lora(m, x, a, b, ids)
    for s in (2.0 ** 60, 2.0 ** -60):
        assert torch.equal(run_lora(m, x * s, a, b, ids), want * s)


def test_lora_offsets_past_32_bits(m):
    """Adapters past 4 GiB, and rows of x and y past 2^31 values."""
    n, r, K, N = 40, 256, 8192, 220000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    g = gen(1)
    b = torch.zeros(n, N, r, dtype=torch.bfloat16, device="cuda")  # 4.5 GB
    a = torch.zeros(n, r, K, dtype=torch.bfloat16, device="cuda")
    b[n - 1, -50:], a[n - 1] = torch.randn(50, r, device="cuda", generator=g).bfloat16(), torch.randn(r, K, device="cuda", generator=g).bfloat16()
    x = torch.randn(2, K, device="cuda", generator=g).bfloat16()
    ids = torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda")
    got = run_lora(m, x, a, b, ids)
    want, size = ref.lora(host64(x[:1]), host64(a[n - 1:]), host64(b[n - 1:, -50:]), np.array([0]))
    assert np.all(np.abs(host64(got[:1, -50:]) - want) <= (K + r + 8) * 2.0 ** -23 * size)
    assert not torch.any(got[0, :-50]) and not torch.any(got[1])
    del b, got
    for T in (4, 70):
        ld = (1 << 31) // (T - 1) // 8 * 8 + 8
        a, b = pool(3, 16, 256, 300, g)
        x, base = torch.randn(T, 256, device="cuda", generator=g).bfloat16(), torch.randn(T, 300, device="cuda", generator=g)
        ids = (torch.arange(T, device="cuda") % 3).to(torch.int32)
        far = torch.empty((T - 1) * ld + 256, dtype=torch.bfloat16, device="cuda")
        y = torch.empty((T - 1) * ld + 300, device="cuda")
        torch.as_strided(far, (T, 256), (ld, 1)).copy_(x)
        torch.as_strided(y, (T, 300), (ld, 1)).copy_(base)
        size = m.moe_lora_workspace_bytes(T, 256, 16)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        m.moe_lora_add(far, m.MOE_X_BF16, ld, a, b, None, None, ids, 3, 16, T, 300, 256, y, ld, y, m.MOE_X_F32, ld, ws, size)
        assert torch.equal(torch.as_strided(y, (T, 300), (ld, 1)), run_lora(m, x, a, b, ids, base=base))
        del far, y


@pytest.mark.parametrize("T,N,K,n,r", [(4097, 300, 288, 5, 16), (70000, 40, 64, 3, 8), (1 << 20, 3, 8, 2, 8)])
def test_lora_prompts(m, T, N, K, n, r):
    """As many tokens as a prompt has, and as many as a call takes: each a copy of one of some tokens."""
    g = gen(T)
    a, b = pool(n, r, K, N, g)
    few = 37 * n
    x, ids = torch.randn(few, K, device="cuda", generator=g).bfloat16(), (torch.arange(few, device="cuda") % (n + 1) - 1).to(torch.int32)
    want, size = ref.lora(host64(x), host64(a), host64(b), ids.cpu().numpy())
    at = torch.randint(0, few, (T,), device="cuda", generator=g)
    at = torch.where(torch.arange(T, device="cuda") % 1000 < 500, at.sort().values, at)  # stretches in order, and not
    got = run_lora(m, x[at], a, b, ids[at].contiguous())
    tol = torch.from_numpy((K + r + 8) * 2.0 ** -23 * size).cuda()
    assert torch.all((got.double() - torch.from_numpy(want).cuda()[at]).abs() <= tol[at])
    first = torch.full((few,), T, device="cuda").scatter_reduce_(0, at, torch.arange(T, device="cuda"), "amin")
    assert torch.equal(got, got[first[at]])  # the same token gives the same bits wherever it stands


# ------------------------------------------- together, streams and graphs


def test_adapters_take_fewer_tokens_than_they_were_made_for(m):
    """The most tokens at once are not those that need the largest workspace: 4160 are split in fewer parts than 4096."""
    from expert_vram_slot_amd.layer import Adapters
    g = gen(41)
    N, K, n, r = 24, 1024, 3, 16
    a = torch.randn(n, r, K, device="cuda", generator=g).bfloat16()
    b = torch.randn(n, N, r, device="cuda", generator=g).bfloat16()
    pool = Adapters(a=a, b=b, T_max=4160)
    for T in (4160, 4096, 1025, 1024, 65, 1):
        x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
        ids = torch.randint(-1, n, (T,), device="cuda", generator=g, dtype=torch.int32)
        base = torch.randn(T, N, device="cuda", generator=g)
        y = pool.add(x, T, ids, base.clone())
        h = torch.einsum("tk,trk->tr", x.double(), a.double()[ids.clamp(min=0).long()])
        size = torch.einsum("tk,trk->tr", x.double().abs(), a.double()[ids.clamp(min=0).long()].abs())
        bb = b.double()[ids.clamp(min=0).long()] * (ids >= 0)[:, None, None]
        want = base.double() + torch.einsum("tr,tnr->tn", h, bb)
        bound = (K + r + 8) * 2.0 ** -23 * (base.double().abs() + torch.einsum("tr,tnr->tn", size, bb.abs()))
        assert torch.all((y.double() - want).abs() <= bound)


def test_a_decode_step_of_many_tenants(m):
    """Two 4-bit layers under a selection rule, the head with each request's adapter, a draw; then the router's training
    step: counts, bias and the gradient of both losses.  Each against its reference on what it was given."""
    import ops_reference
    import synth
    from expert_vram_slot_amd.layer import Adapters, DecodeHead, SlotStack
    E, k, H, I, S, T, V, group = 16, 4, 256, 128, 16, 5, 3001, 64
    base = synth.config_seed("c4")
    layers = []
    for n in range(2):
        store = synth.slabs(synth.W_Q4B32, base, n, 0, E, H, I, 0.05)
        pinned = torch.empty(store.shape, dtype=torch.uint8, pin_memory=True)
        pinned.copy_(torch.from_numpy(store))
        G = synth.normal(synth.key(base, synth.TAG_G, n, 0), (E, H), 0.5, synth.X_BF16)
        layers.append(dict(host_store=pinned, slot_store=torch.from_numpy(store).cuda(), bias=torch.zeros(E, device="cuda"),
                           G=torch.from_numpy(G.view(np.int16)).cuda(),
                           resident=torch.arange(S, dtype=torch.int32, device="cuda")))
    rule = dict(score="sigmoid", groups=4, groups_kept=2, group_top=2, scale=2.5)
    stack = SlotStack(E=E, k=k, H=H, I=I, S=S, w_type=synth.W_Q4B32, T_max=8, layers=layers, n_threads=1,
                      select=m.select_rule(**rule))
    g = gen(6)
    wq = torch.randint(0, 256, (V, H // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = (0.003 + 0.004 * torch.rand(V, H // group, device="cuda", generator=g)).half()
    a, b = pool(3, 16, H, V, g)
    lora_scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    head = DecodeHead(H=H, V=V, wq=wq, scales=scales, group=group, T_max=8, adapters=Adapters(a=a, b=b, T_max=8, scale=lora_scale))
    u = torch.rand(T, device="cuda", generator=g)
    adapter_ids = torch.tensor([2, -1, 0, 1, 2], dtype=torch.int32, device="cuda")

    def check_layer(l, L, x, y):
        z = L.logits[:T * E].view(T, E)
        bias = L.bias.clone()
        want_ids, want_w, _ = ref.select(host64(z), k, bias=host64(bias), **plain(rule))
        picks = L.ids[:T * k].view(T, k)
        np.testing.assert_array_equal(picks.cpu().numpy(), want_ids)
        assert np.all(np.abs(host64(L.w[:T * k].view(T, k)) - want_w) <= (2.0 ** -24 + 2.0 ** -45) * want_w)
        bal = L.balance(T)
        dz = L.balance_grad(T, torch.tensor([1.0, 0.1], device="cuda"))
        dw = torch.randn(T, k, device="cuda", generator=g)
        both = L.select_grad(T, dw, dz)
        part, size = ref.select_grad(host64(z), want_ids, host64(dw), rule["score"], True, rule["scale"])
        want = part + host64(dz)
        assert np.all(np.abs(host64(both) - want) <= 3 * DS(E) * size + 2.0 ** -22 * (np.abs(want) + np.abs(part)))
        assert np.all(np.abs(host64(L.select_grad(T, dw)) - part) <= 3 * DS(E) * size + 2.0 ** -22 * np.abs(part))
        L.balance_bias(0.01)
        want_bias = ref.bias_balance(bal["counts"].cpu().numpy()[None], bias.cpu().numpy()[None], 0.01)[0]
        np.testing.assert_array_equal(L.bias.cpu().numpy(), want_bias)

    for step in range(3):
        x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
        h = stack.step(x, T, host_pass=False, on_layer=check_layer)
        ids, prob = head.step(h, T, u, adapter_ids=adapter_ids)
        torch.cuda.synchronize()
        shared, size = ops_reference.linear_q4(host64(h), wq.cpu().numpy(), scales.cpu().numpy(), group)
        want, size2 = ref.lora(host64(h), host64(a), host64(b), adapter_ids.cpu().numpy(), None, host64(lora_scale))
        got = host64(head.logits_buf[:T])
        tol = (2 * 128 + H / 32 + 8) * 2.0 ** -23 * size + (H + 16 + 8) * 2.0 ** -23 * (size2 + size)
        assert np.all(np.abs(got - shared - want) <= tol)
        for t in range(T):
            i, q, _ = ops_reference.sample_row(got[t], float(u[t]))
            assert int(ids[t]) == i and abs(float(prob[t]) - q) <= 2.0 ** -24 * q + V * 2.0 ** -50
        plain_logits = head.logits(h, T).clone()  # no adapters: the shared product alone
        assert np.all(np.abs(host64(plain_logits) - shared) <= (2 * 128 + H / 32 + 8) * 2.0 ** -23 * size)
        assert torch.equal(plain_logits[1], torch.from_numpy(got[1]).float().cuda())


def test_a_layer_under_a_rule_with_padding_and_given_picks(m):
    """A padded batch's tokens pick nothing and get 0; given picks get the rule's weights; the host pass joins in."""
    import synth
    from expert_vram_slot_amd.layer import SlotLayer
    E, k, H, I, S, T = 16, 4, 256, 128, 8, 6
    base = synth.config_seed("c4")
    store = synth.slabs(synth.W_Q4B32, base, 0, 0, E, H, I, 0.05)
    pinned = torch.empty(store.shape, dtype=torch.uint8, pin_memory=True)
    pinned.copy_(torch.from_numpy(store))
    G = synth.normal(synth.key(base, synth.TAG_G, 0, 0), (E, H), 0.5, synth.X_BF16)
    a = dict(E=E, k=k, H=H, I=I, S=S, w_type=synth.W_Q4B32, T_max=8, policy="static", host_store=pinned,
             slot_store=torch.from_numpy(store[:S]).cuda(), G=torch.from_numpy(G.view(np.int16)).cuda(), n_threads=1)
    L = SlotLayer(**a, select=m.select_rule("softmax"))
    same = SlotLayer(**a)  # moe_route's own rule is the renormalised softmax
    for layer in (L, same):
        layer.init_cache(torch.arange(S, dtype=torch.int32, device="cuda"))
    x = torch.randn(T, H, device="cuda", generator=gen(2)).bfloat16()
    want = same.step(x, T).clone()
    assert torch.equal(L.step(x, T), want)
    mask = torch.tensor([1, 0, 1, 1, 0, 1], dtype=torch.uint8, device="cuda")
    for host_pass in (False, True):
        got = L.step(x, T, mask=mask, host_pass=host_pass)
        torch.cuda.synchronize()
        assert torch.all(got[mask == 0] == 0)
        if host_pass:
            assert torch.equal(got[mask == 1], want[mask == 1])
    assert torch.all(L.ids[:T * k].view(T, k)[mask == 0] == -1)
    assert not torch.any(L.select_grad(T, torch.ones(T, k, device="cuda"))[mask == 0])
    picks = torch.randint(0, E, (T, k), device="cuda", generator=gen(3)).to(torch.int32)
    L.step(x, T, ids_in=picks, host_pass=False)
    _, w, _ = ref.select(host64(L.logits[:T * E].view(T, E)), k, ids_in=picks.cpu().numpy())
    assert np.all(np.abs(host64(L.w[:T * k].view(T, k)) - w) <= (2.0 ** -24 + 2.0 ** -45) * w)


def _whole_path(m, T, N, K, seed):
    """Buffers and a call of every operator; returns (call, inputs to refill, outputs)."""
    g = gen(seed)
    E, k, n, r, L = 96, 6, 5, 24, 3
    Z = 16 * T
    z, bias = torch.randn(Z, E, device="cuda", generator=g), 0.01 * torch.randn(L, E, device="cuda", generator=g)
    ids, w = torch.empty(Z, k, dtype=torch.int32, device="cuda"), torch.empty(Z, k, device="cuda")
    dw, dz = torch.randn(Z, k, device="cuda", generator=g), torch.empty_like(z)
    dz2 = torch.empty_like(z)
    counts, out = torch.randint(0, 50, (L, E), device="cuda", generator=g).to(torch.int32), torch.empty(L, E, device="cuda")
    a, b = pool(n, r, K, N, g)
    x, aid = torch.randn(T, K, device="cuda", generator=g).bfloat16(), some_ids(T, n, "mixed", g)
    base, y = torch.randn(T, N, device="cuda", generator=g), torch.empty(T, N, device="cuda")
    size = m.moe_lora_workspace_bytes(T, K, r)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    grouped = m.select_rule("sigmoid", groups=8, groups_kept=3, group_top=2)
    raw = m.select_rule("softmax", renorm=False)

    def call(stream=None):
        m.moe_route_select(z, m.MOE_X_F32, bias, None, None, Z, E, k, grouped, ids, w, stream)
        m.moe_route_select_bwd(z, m.MOE_X_F32, ids, dw, Z, E, k, grouped, None, dz, stream)
        m.moe_route_select_bwd(z, m.MOE_X_F32, ids, dw, Z, E, k, raw, dz, dz2, stream)
        m.moe_bias_balance(counts, bias, L, E, 0.01, out, stream)
        m.moe_lora_add(x, m.MOE_X_BF16, K, a, b, None, None, aid, n, r, T, N, K, base, N, y, m.MOE_X_F32, N, ws, size, stream)

    return call, (z, x, base), (ids, w, dz, dz2, out, y)


@pytest.mark.parametrize("T,N", [(1, 2001), (20, 9000), (300, 1500)])
def test_captured_and_replayed_with_eager_calls_between(m, T, N):
    call, inputs, outputs = _whole_path(m, T, N, 512, 1)
    other, _, _ = _whole_path(m, T + 3, N + 77, 256, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(4):
        g = gen(50 + rep)
        for t in inputs:
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
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
    paths = [_whole_path(m, T, 9000, 512, T) for T in (6, 300)]
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


# ------------------------------------------- groups larger than a wave's registers


LARGE_GROUPS = [  # T, E, k, groups, kept, top: more than 64 experts a lane, and 64
    (5, 2145, 8, 33, 5, 2), (9, 4095, 8, 3, 2, 2), (7, 4000, 10, 10, 4, 1), (3, 2565, 3, 5, 5, 2), (4, 2210, 32, 34, 20, 1),
    (2, 4080, 17, 48, 1, 2), (5, 2112, 8, 33, 5, 2)]


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
@pytest.mark.parametrize("T,E,k,groups,kept,top", LARGE_GROUPS)
def test_select_large_groups(m, T, E, k, groups, kept, top, rule, with_bias, zt):
    """Ordinary logits, far ones (700 and more is beyond what exp takes without the maximum off), nothing open, padding."""
    rule = dict(rule, groups=groups, groups_kept=kept, group_top=top)
    g = gen(E + k)
    z = torch.cat([logits(T, E, T * E + k), 4.0 * logits(2, E, 1) + 800.0, logits(1, E, 2) - 900.0, special_rows(E, g)]).to(DT[zt])
    bias = 0.001 * torch.randint(-80, 81, (E,), device="cuda", generator=g).float() if with_bias else None
    ids, _ = check_select(m, z, k, rule, bias)
    check_grad(m, z, ids, torch.randn(*ids.shape, device="cuda", generator=g), rule)
    check_select(m, z, k, rule, bias, (torch.arange(len(z), device="cuda") % 3 != 1).to(torch.uint8))


@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r['score']}{'' if r.get('renorm', True) else '_raw'}")
@pytest.mark.parametrize("E,k,groups", [(2145, 8, 33), (4095, 20, 3)])
def test_select_large_groups_of_many_tokens(m, E, k, groups, rule):
    """A wave takes several tokens: each gets its own sum and picks.  Tokens are copies of some, which are checked."""
    rule = dict(rule, groups=groups, groups_kept=2, group_top=2)
    g = gen(E)
    some = logits(37, E, 5)
    at = torch.randint(0, 37, (16500,), device="cuda", generator=g)
    bias = 0.001 * torch.randint(-80, 81, (E,), device="cuda", generator=g).float()
    want_ids, want_w = check_select(m, some, k, rule, bias)
    ids, w = run_select(m, some[at], k, rule, bias)
    assert torch.equal(ids, want_ids[at]) and torch.equal(w, want_w[at])


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept", [(8, 8, 4, 4), (8, 3, 4, 3), (96, 6, 3, 2), (288, 8, 8, 4), (288, 32, 8, 8), (2145, 8, 33, 30)])
def test_select_groups_of_lowest_biases(m, E, k, groups, kept, score, zt):
    """Two biases of the type's lowest value add up to more than fp32 holds; their group is open all the same, and stands
    behind the others, before those with nothing open."""
    g, gs, low = gen(E + k), E // groups, torch.finfo(torch.float32).min
    z = logits(6, E, E, zt)
    z[5] = 0
    for group_top in (1, 2):
        rule = dict(score=score, groups=groups, groups_kept=kept, group_top=group_top)
        for masked in ([0], [0, groups - 1], range(groups), range(1, groups), range(groups - 1)):
            for value in (low, -2e38, -low):
                bias = 0.001 * torch.randint(-80, 81, (E,), device="cuda", generator=g).float()
                for i in masked:
                    bias[i * gs:(i + 1) * gs] = value
                check_select(m, z, k, rule, bias)
                bias[gs:2 * gs] = -float("inf")  # one group is closed
                bias[gs * (groups - 1)] = low    # and one has a single expert as low as this
                check_select(m, z, k, rule, bias)


@pytest.mark.parametrize("T", [1, 70, 1200])
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_lora_without_base_or_adapter_is_zero(m, T, yt):
    """No base is a base of zeros, of a positive sign in every column."""
    a, b = pool(2, 16, 64, 200, gen(1))
    ids = (torch.arange(T, device="cuda") % 3 - 1).to(torch.int32)
    ranks = torch.tensor([16, 0], dtype=torch.int32, device="cuda")
    got = run_lora(m, torch.randn(T, 64, device="cuda").bfloat16(), a, b, ids, ranks, None, None, yt)
    without = got[ids != 0].contiguous()
    assert not torch.any(without.view(torch.int32 if yt == "f32" else torch.int16))


def test_a_stack_keeps_its_layers_counts_apart(m):
    """A bias moves by its own layer's counts of the last step, or not at all."""
    import synth
    from expert_vram_slot_amd.layer import SlotStack
    E, k, H, I, T = 16, 4, 256, 128, 5
    base = synth.config_seed("c4")
    layers = []
    for n in range(2):
        store = synth.slabs(synth.W_Q4B32, base, n, 0, E, H, I, 0.05)
        pinned = torch.empty(store.shape, dtype=torch.uint8, pin_memory=True)
        pinned.copy_(torch.from_numpy(store))
        G = synth.normal(synth.key(base, synth.TAG_G, n, 0), (E, H), 0.5, synth.X_BF16)
        layers.append(dict(host_store=pinned, slot_store=torch.from_numpy(store).cuda(), bias=torch.zeros(E, device="cuda"),
                           G=torch.from_numpy(G.view(np.int16)).cuda(), resident=torch.arange(E, dtype=torch.int32, device="cuda")))
    stack = SlotStack(E=E, k=k, H=H, I=I, S=E, w_type=synth.W_Q4B32, T_max=8, layers=layers, n_threads=1, select=m.select_rule())
    x = torch.randn(T, H, device="cuda", generator=gen(6)).bfloat16()
    stack.step(x, T, host_pass=False, on_layer=lambda l, L, x_l, y_l: L.balance(T) if l == 0 else None)
    with pytest.raises(AssertionError, match="last step"):  # layer 1's step came behind the counts
        stack.layer.balance_bias(0.01)
    counts = stack.layer.balance(T)["counts"].cpu().numpy()
    with pytest.raises(AssertionError, match="layer 1's, the bias is layer 0's"):
        stack.bind(0).balance_bias(0.01)
    stack.bind(1).balance_bias(0.01)
    assert not torch.any(layers[0]["bias"])
    np.testing.assert_array_equal(layers[1]["bias"].cpu().numpy(), ref.bias_balance(counts[None], np.zeros((1, E), np.float32), 0.01)[0])


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("E,groups", [(8, 1), (8, 4), (64, 1), (288, 1), (288, 8), (512, 16)])
def test_select_border_among_equals_near_others(m, E, groups, zt):
    """The last pick lies among experts of one logit and one choice, and others, less than the fp32 sum's error away, on
    either side of them: whether a sum in double is needed is not decided by the equals alone."""
    g, borders = gen(E + groups), 0
    for equals in (torch.finfo(torch.float32).min, -60.0, 0.25, 2.0):
        for turn in range(6):
            z = logits(1, E, 7 * E + turn, zt)
            order = torch.randperm(E, device="cuda", generator=g).cpu().numpy()
            same, others = order[:min(E // 2, 8)], order[min(E // 2, 8):min(E, 24)]
            z[0, torch.from_numpy(same).cuda()] = equals
            s = ref.scores(host64(z), "softmax")[0]
            bias = np.full(E, -2.0, np.float32)  # the rest are far behind
            bias[same], bias[others] = (0.5 - s[same]).astype(np.float32), (0.5 - s[others]).astype(np.float32)
            ahead = int((s[others] + bias[others] > s[same[0]] + np.float64(bias[same[0]])).sum())
            for k in sorted({1, ahead + 1, ahead + len(same) // 2}):
                borders += len(others) > ahead
                check_select(m, z, k, dict(score="softmax", groups=groups, renorm=turn % 2 == 0), torch.from_numpy(bias).cuda())
    assert borders > 20


@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("E,groups", [(8, 1), (8, 4), (64, 1), (288, 1), (288, 8), (512, 16)])
def test_select_border_before_experts_of_large_scores(m, E, groups, zt):
    """Experts of small scores, that a sum's error hardly moves, stand at the border next to one another; behind them, by
    places, but within that error, stand some of large scores."""
    g, behind = gen(E + groups), 0
    for turn in range(40):
        z = logits(1, E, 9 * E + turn, zt) - 9.0
        order = torch.randperm(E, device="cuda", generator=g).cpu().numpy()
        large, small = order[:2], order[2:min(E, 24)]
        z[0, torch.from_numpy(large).cuda()] = logits(1, 2, 5 * E + turn, zt)[0]
        s = ref.scores(host64(z), "softmax")[0]
        bias = np.full(E, -2.0, np.float32)
        bias[large], bias[small] = (0.5 - s[large]).astype(np.float32), (0.5 - s[small]).astype(np.float32)
        c = s + bias.astype(np.float64)
        places = np.nonzero(np.isin(np.argsort(-c), large))[0]  # of the two of large scores
        for k in sorted({1, int(places[0]) + 1, int(places[1]) + 1, max(1, int(places[1]) - 1)}):
            behind += 0 <= places[0] - k <= 8
            check_select(m, z, k, dict(score="softmax", groups=groups, renorm=turn % 2 == 0), torch.from_numpy(bias).cuda())
    assert behind > 5
