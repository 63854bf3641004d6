"""moe_route_select, moe_bias_balance and moe_lora_add without a GPU: refusals
and workspace sizes (nothing is launched on those paths), and the references of
the GPU tests against brute force, closed forms and differences."""
import ctypes
import itertools

import numpy as np
import pytest

import select_lora_reference as ref


@pytest.fixture(scope="module")
def mlib():
    import os

    from expert_vram_slot_amd import build as b
    if not os.path.exists(b.LIB):
        b.build()
    import expert_vram_slot_amd as m
    m.lib()
    return m


# ------------------------------------------------------------- refusals

LOGITS = dict(x=16, x_dtype=1, G=16, T=4, H=64, E=8, logits=16)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), "ARG"), (dict(G=None), "ARG"), (dict(logits=None), "ARG"), (dict(T=-1), "ARG"), (dict(H=0), "ARG"),
    (dict(E=0), "ARG"), (dict(x_dtype=2), "DTYPE"), (dict(E=4097), "SHAPE"), (dict(H=32776), "SHAPE"),
    (dict(H=16388, x_dtype=0), "SHAPE"), (dict(x=8), "ALIGN"), (dict(G=8), "ALIGN"), (dict(H=60), "ALIGN"),
    (dict(H=66, x_dtype=0), "ALIGN"),
])
def test_route_logits_refuses(mlib, change, code):
    a = dict(LOGITS, **change)
    rc = mlib.lib().moe_route_logits(*[a[n] for n in LOGITS], None)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_route_logits:")


RULE = dict(score=1, groups=4, groups_kept=2, group_top=2, renorm=1, scale=2.5)
SELECT = dict(z=16, z_dtype=0, bias=16, mask=16, ids_in=None, T=4, E=16, k=4, rule=RULE, ids=16, w=16)
GRAD = dict(z=16, z_dtype=0, ids=16, dw=16, T=4, E=16, k=4, rule=RULE, dz_add=16, dz=16)
BAD_RULES = [
    (dict(score=2), "ARG"), (dict(score=-1), "ARG"), (dict(groups=0), "ARG"), (dict(groups_kept=0), "ARG"),
    (dict(groups_kept=5), "ARG"), (dict(group_top=0), "ARG"), (dict(group_top=3), "ARG"), (dict(scale=np.inf), "ARG"),
    (dict(scale=np.nan), "ARG"), (dict(groups=3), "SHAPE"), (dict(groups=5, groups_kept=2), "SHAPE"),
    (dict(groups_kept=1, groups=8), "SHAPE"),  # two experts for four picks
]
BAD_BOTH = [
    (dict(z=None), "ARG"), (dict(rule=None), "ARG"), (dict(T=-1), "ARG"), (dict(E=0), "ARG"), (dict(k=0), "ARG"),
    (dict(z_dtype=2), "DTYPE"), (dict(E=4100), "SHAPE"), (dict(k=17), "SHAPE"), (dict(E=64, k=33), "SHAPE"),
    (dict(k=9), "SHAPE"), (dict(T=(1 << 24) + 1), "SHAPE"), (dict(E=1040, rule=dict(RULE, groups=65)), "SHAPE"),
    (dict(z=20), "ALIGN"), (dict(ids=18), "ALIGN"),
] + [(dict(rule=dict(RULE, **c)), code) for c, code in BAD_RULES]


def _call(mlib, name, base, change):
    a = dict(base, **change)
    if a["rule"] is not None:
        a["rule"] = ctypes.byref(mlib.SelectRule(*[a["rule"][n] for n in RULE]))
    return getattr(mlib.lib(), name)(*[a[n] for n in base], None)


@pytest.mark.parametrize("change,code", BAD_BOTH + [(dict(w=None), "ARG"), (dict(ids=None), "ARG"), (dict(w=17), "ALIGN"),
                                                    (dict(ids_in=18), "ALIGN"), (dict(bias=18), "ALIGN")])
def test_select_refuses(mlib, change, code):
    rc = _call(mlib, "moe_route_select", SELECT, change)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_route_select:")


@pytest.mark.parametrize("change,code", BAD_BOTH + [(dict(ids=None), "ARG"), (dict(dw=None), "ARG"), (dict(dz=None), "ARG"),
                                                    (dict(dz=8), "ALIGN"), (dict(dz_add=8), "ALIGN"), (dict(dw=2), "ALIGN")])
def test_select_grad_refuses(mlib, change, code):
    rc = _call(mlib, "moe_route_select_bwd", GRAD, change)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_route_select_bwd:")


def test_select_of_no_tokens(mlib):
    nothing = dict(z=None, ids=None, T=0)
    assert _call(mlib, "moe_route_select", SELECT, dict(nothing, w=None)) == mlib.MOE_OK
    assert _call(mlib, "moe_route_select_bwd", GRAD, dict(nothing, dw=None, dz=None)) == mlib.MOE_OK


BIAS = dict(counts=16, bias=16, L=2, E=8, rate=0.001, bias_out=16)


@pytest.mark.parametrize("change,code", [
    (dict(counts=None), "ARG"), (dict(bias=None), "ARG"), (dict(bias_out=None), "ARG"), (dict(L=0), "ARG"),
    (dict(E=0), "ARG"), (dict(rate=-0.1), "ARG"), (dict(rate=np.inf), "ARG"), (dict(rate=np.nan), "ARG"),
    (dict(E=4097), "SHAPE"), (dict(L=65536), "SHAPE"),
])
def test_bias_balance_refuses(mlib, change, code):
    a = dict(BIAS, **change)
    rc = mlib.lib().moe_bias_balance(*[a[n] for n in BIAS], None)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_bias_balance:")


LORA = dict(x=16, x_dtype=1, ldx=64, a=16, b=16, ranks=16, scale=16, ids=16, n=3, r=16, T=4, N=9, K=64, base=32, ldb=12,
            y=64, y_dtype=0, ldy=9, ws=16, ws_bytes=1 << 30)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), "ARG"), (dict(a=None), "ARG"), (dict(b=None), "ARG"), (dict(ids=None), "ARG"), (dict(y=None), "ARG"),
    (dict(ws=None), "ARG"), (dict(T=-1), "ARG"), (dict(N=0), "ARG"), (dict(K=0), "ARG"), (dict(n=0), "ARG"),
    (dict(r=0), "ARG"), (dict(ldx=56), "ARG"), (dict(ldb=8), "ARG"), (dict(ldy=8), "ARG"), (dict(base=64), "ARG"),
    (dict(ws_bytes=15), "ARG"), (dict(ldx=-64), "ARG"),
    (dict(x_dtype=2), "DTYPE"), (dict(y_dtype=7), "DTYPE"),
    (dict(K=60), "SHAPE"), (dict(r=12), "SHAPE"), (dict(r=264), "SHAPE"), (dict(n=65537), "SHAPE"),
    (dict(T=(1 << 20) + 1), "SHAPE"), (dict(N=(1 << 22) + 1, ldb=1 << 23, ldy=1 << 23), "SHAPE"),
    (dict(K=(1 << 22) + 8, ldx=1 << 23), "SHAPE"), (dict(ldx=1 << 41), "SHAPE"), (dict(ldy=1 << 41), "SHAPE"),
    (dict(ldb=1 << 41), "SHAPE"),
    (dict(x=8), "ALIGN"), (dict(a=8), "ALIGN"), (dict(b=24), "ALIGN"), (dict(ws=8), "ALIGN"), (dict(ldx=68), "ALIGN"),
    (dict(ldx=66, x_dtype=0), "ALIGN"), (dict(base=34), "ALIGN"), (dict(y=66), "ALIGN"), (dict(y=65, y_dtype=1), "ALIGN"),
    (dict(ids=18), "ALIGN"), (dict(ranks=18), "ALIGN"), (dict(scale=18), "ALIGN"),
])
def test_lora_refuses(mlib, change, code):
    a = dict(LORA, **change)
    rc = mlib.lib().moe_lora_add(*[a[n] for n in LORA], None)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_lora_add:")


def test_lora_of_no_tokens_and_workspace(mlib):
    a = dict(LORA, T=0, x=None, ids=None, y=None, base=None)
    assert mlib.lib().moe_lora_add(*[a[n] for n in LORA], None) == mlib.MOE_OK
    assert mlib.moe_lora_workspace_bytes(0, 64, 8) > 0
    assert mlib.moe_lora_workspace_bytes(64, 64, 16) >= mlib.moe_lora_workspace_bytes(1, 64, 16)
    for bad in ((-1, 64, 8), (1, 0, 8), (1, 64, 0), (1, 64, 257), ((1 << 20) + 1, 64, 8)):
        assert mlib.moe_lora_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("K", [8, 256, 520, 1000, 1024, 8192])
def test_a_workspace_is_enough_for_fewer_tokens(mlib, K):
    """A caller makes it once, for the most tokens."""
    sizes = [mlib.moe_lora_workspace_bytes(T, K, 24) for T in [*range(0, 200), *range(1000, 18000, 8), 1 << 17, 1 << 20]]
    assert all(x <= y for x, y in zip(sizes, sizes[1:]))



def test_binding_raises_with_the_reason(mlib):
    with pytest.raises(mlib.MoeError) as e:
        mlib.moe_route_select(16, 0, None, None, None, 1, 10, 2, mlib.select_rule(groups=4), 16, 16, stream=0)
    assert e.value.code == mlib.MOE_E_SHAPE and "10 experts in 4 groups" in str(e.value)
    with pytest.raises(mlib.MoeError):
        mlib.moe_route_select_bwd(16, 0, 16, 16, 1, 8, 2, mlib.select_rule(score=7), None, 16, stream=0)
    with pytest.raises(mlib.MoeError):
        mlib.moe_route_logits(16, 0, 16, 1, 63, 8, 16, stream=0)
    with pytest.raises(mlib.MoeError):
        mlib.moe_bias_balance(16, 16, 1, 8, -1.0, 16, stream=0)
    with pytest.raises(mlib.MoeError):
        mlib.moe_lora_add(16, 1, 64, 16, 16, None, None, 16, 1, 12, 1, 8, 64, None, 0, 16, 0, 8, 16, 1 << 20, stream=0)


def test_select_rule_defaults(mlib):
    r = mlib.select_rule()
    assert (r.score, r.groups, r.groups_kept, r.group_top, r.renorm, r.scale) == (0, 1, 1, 1, 1, 1.0)
    r = mlib.select_rule("sigmoid", groups=8, group_top=2, renorm=False, scale=2.5)
    assert (r.score, r.groups, r.groups_kept, r.group_top, r.renorm, r.scale) == (1, 8, 8, 2, 0, 2.5)


def _layer_after_a_step(T, m):
    """The part of a SlotLayer that its gradients look at, on the CPU, as a step of T tokens leaves it."""
    import torch

    from expert_vram_slot_amd.layer import SlotLayer
    L = SlotLayer.__new__(SlotLayer)
    L.E, L.k, L.T_max, L.stats_out = 8, 2, 4, None
    L.logits, L.ids, L.bias = torch.zeros(32), torch.zeros(8, dtype=torch.int32), torch.zeros(8)
    L.steps, L.step_T, L.captured, L.balanced = 1, T, False, None
    L.select, L.route_flags = m.select_rule(), 0
    return L


@pytest.mark.parametrize("change", [dict(T=3), dict(T=5), dict(dw="f64"), dict(dw="short"), dict(dw="strided"),
                                    dict(dw="elsewhere"), dict(dw=None), dict(dz_add="short"), dict(dz_add="bf16"),
                                    dict(rule=None)])
def test_layer_select_grad_refuses(mlib, change):
    torch = pytest.importorskip("torch")
    L = _layer_after_a_step(2, mlib)
    bad = {"f64": torch.zeros(2, 2, dtype=torch.float64), "short": torch.zeros(3), "strided": torch.zeros(2, 4)[:, ::2],
           "elsewhere": torch.zeros(2, 2, device="meta"), "bf16": torch.zeros(2, 8, dtype=torch.bfloat16)}
    a = dict(T=2, dw=torch.zeros(2, 2))
    for n, v in change.items():
        if n == "rule":
            L.select = None
        else:
            a[n] = bad[v] if isinstance(v, str) else v
    with pytest.raises(AssertionError):
        L.select_grad(**a)


@pytest.mark.parametrize("change", ["no balance", "no bias", "f64", "short", "strided"])
def test_layer_balance_bias_refuses(mlib, change):
    torch = pytest.importorskip("torch")
    L = _layer_after_a_step(2, mlib)
    L.stats_out = None if change == "no balance" else dict(counts=torch.zeros(8, dtype=torch.int32))
    L.bias = {"no bias": None, "f64": torch.zeros(8, dtype=torch.float64), "short": torch.zeros(7),
              "strided": torch.zeros(16)[::2]}.get(change, L.bias)
    with pytest.raises(AssertionError):
        L.balance_bias(0.001)


@pytest.mark.parametrize("change", [dict(mask="i64"), dict(mask="short"), dict(select=None), dict(ids_in=True),
                                    dict(flags=1, mask=None)])
def test_layer_step_refuses_masks(mlib, change):
    torch = pytest.importorskip("torch")
    L = _layer_after_a_step(2, mlib)
    a = dict(x=torch.zeros(2, 64), T=2, mask=torch.ones(2, dtype=torch.uint8))
    bad = {"i64": torch.ones(2, dtype=torch.int64), "short": torch.ones(1, dtype=torch.uint8)}
    for n, v in change.items():
        if n == "select":
            L.select = None
        elif n == "flags":
            L.route_flags = v
        elif n == "ids_in":
            a[n] = torch.zeros(2, 2, dtype=torch.int32)
        else:
            a[n] = bad.get(v, v)
    with pytest.raises(AssertionError):
        L.step(**a)


POOL = dict(a=(3, 16, 64), b=(3, 8, 16))


def _pool(**change):
    import torch

    from expert_vram_slot_amd.layer import Adapters
    a = dict(a=torch.zeros(POOL["a"], dtype=torch.bfloat16), b=torch.zeros(POOL["b"], dtype=torch.bfloat16), T_max=4)
    a.update(change)
    return Adapters(**a)


@pytest.mark.parametrize("change", ["b rows", "b ranks", "f16", "strided", "ranks", "ranks type", "scale", "elsewhere",
                                    "r", "T_max"])
def test_adapters_refuse(mlib, change):
    torch = pytest.importorskip("torch")
    _pool()
    bf = dict(dtype=torch.bfloat16)
    bad = {"b rows": dict(b=torch.zeros(2, 8, 16, **bf)), "b ranks": dict(b=torch.zeros(3, 8, 8, **bf)),
           "f16": dict(a=torch.zeros(POOL["a"], dtype=torch.float16)),
           "strided": dict(a=torch.zeros(3, 16, 128, **bf)[:, :, ::2]),
           "ranks": dict(ranks=torch.zeros(2, dtype=torch.int32)), "ranks type": dict(ranks=torch.zeros(3, dtype=torch.int64)),
           "scale": dict(scale=torch.zeros(3, dtype=torch.float64)),
           "elsewhere": dict(b=torch.zeros(3, 8, 16, device="meta", **bf)),
           "r": dict(a=torch.zeros(3, 264, 64, **bf), b=torch.zeros(3, 8, 264, **bf)), "T_max": dict(T_max=1 << 21)}
    with pytest.raises(AssertionError):
        _pool(**bad[change])


@pytest.mark.parametrize("change", [dict(T=5), dict(x="f32"), dict(x="short"), dict(x="columns"), dict(y="bf16"),
                                    dict(y="short"), dict(y="columns"), dict(ids="i64"), dict(ids="short"), dict(ids=None),
                                    dict(y="elsewhere")])
def test_adapters_add_refuses(mlib, change):
    torch = pytest.importorskip("torch")
    pool = _pool()
    bf = dict(dtype=torch.bfloat16)
    bad = dict(x={"f32": torch.zeros(2, 64), "short": torch.zeros(127, **bf), "columns": torch.zeros(2, 128, **bf)[:, ::2]},
               y={"bf16": torch.zeros(2, 8, **bf), "short": torch.zeros(15), "columns": torch.zeros(2, 16)[:, ::2],
                  "elsewhere": torch.zeros(2, 8, device="meta")},
               ids={"i64": torch.zeros(2, dtype=torch.int64), "short": torch.zeros(1, dtype=torch.int32), None: None})
    a = dict(x=torch.zeros(2, 64, **bf), T=2, ids=torch.zeros(2, dtype=torch.int32), y=torch.zeros(2, 8))
    for n, v in change.items():
        a[n] = v if n == "T" else bad[n][v]
    with pytest.raises(AssertionError):
        pool.add(**a)


def test_decode_head_refuses_adapters(mlib):
    torch = pytest.importorskip("torch")
    from expert_vram_slot_amd.layer import DecodeHead
    a = dict(H=64, V=8, wq=torch.zeros(8, 32, dtype=torch.uint8), scales=torch.zeros(8, 2, dtype=torch.float16), group=32,
             T_max=2, device="cpu")
    head = DecodeHead(**a, adapters=_pool())
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(AssertionError):
        head.logits(x, 2, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(AssertionError):
        DecodeHead(**a).logits(x, 2, torch.zeros(2, dtype=torch.int32))
    for bad in (dict(T_max=1), dict(y_dtype=mlib.MOE_X_BF16), dict(x_dtype=mlib.MOE_X_F32),
                dict(b=torch.zeros(3, 9, 16, dtype=torch.bfloat16))):
        with pytest.raises(AssertionError):
            DecodeHead(**a, adapters=_pool(**bad))


# ------------------------------------------------------------ references


@pytest.mark.parametrize("seed", range(30))
def test_reference_choice_against_brute_force(seed):
    """Every set of groups and every order of experts tried against the definition."""
    rng = np.random.default_rng(seed)
    groups = int(rng.choice([1, 2, 3]))
    gs = int(rng.integers(1, 4)) if groups > 1 else int(rng.integers(1, 7))
    E, kept, top = groups * gs, int(rng.integers(1, groups + 1)), int(rng.integers(1, 3))
    z = rng.integers(-2, 3, E).astype(np.float64)  # ties are common
    z[rng.random(E) < 0.15] = -np.inf
    bias = rng.integers(-2, 3, E) * 0.25 if seed % 2 else None
    if bias is not None:
        bias[rng.random(E) < 0.1] = -np.inf
    s = ref.scores(z[None], "sigmoid")[0]
    k = int(rng.integers(1, kept * gs + 1))
    got = ref.choose(z, s, k, bias, groups, kept, top)
    c = s + (0 if bias is None else bias)
    is_open = [e for e in range(E) if z[e] > -np.inf and (bias is None or bias[e] > -np.inf)]
    best, best_value = (), ()
    for n in range(kept, -1, -1):  # of the sets of groups with something open, the best by value, then by lower groups
        for chosen in itertools.combinations(range(groups), n):
            members = [[e for e in is_open if e // gs == g] for g in chosen]
            if not all(members):
                continue
            value = sorted((sum(sorted((c[e] for e in m), reverse=True)[:top]) for m in members), reverse=True)
            if len(chosen) > len(best) or (len(chosen) == len(best) and tuple(value) > tuple(best_value)):
                best, best_value = chosen, value
    if groups == 1:
        best = (0,)
    left = [e for e in is_open if e // gs in best]
    want = next((list(p) for n in (min(k, len(left)),) for p in itertools.permutations(left, n)
                 if all((c[a], z[a], -a) > (c[b], z[b], -b) for a, b in zip(p, p[1:]))
                 and all((c[p[-1]], z[p[-1]], -p[-1]) >= (c[e], z[e], -e) for e in left if e not in p)), [])
    assert list(got) == want + [-1] * (k - len(want))


def test_reference_select_hand_cases():
    z = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    ids, w, s = ref.select(z, 2, renorm=False, scale=2.0)
    assert list(ids[0]) == [1, 2] and w[0] == pytest.approx([1.0, 0.5])
    ids, w, _ = ref.select(z, 2)
    assert w[0] == pytest.approx([2 / 3, 1 / 3])
    # a bias on the scores moves the choice, not the weights: 1/8 + 1/2 against 4/8 and 2/8
    ids, w, _ = ref.select(z, 2, bias=np.array([0, 0, 0, 0.5]), renorm=False)
    assert list(ids[0]) == [3, 1] and w[0] == pytest.approx([1 / 8, 1 / 2])
    # groups of two: 1 + 4 against 2 + 1 eighths; the best alone: 4 against 2
    assert list(ref.select(z, 2, groups=2, kept=1, top=2)[0][0]) == [1, 0]
    assert list(ref.select(z, 1, groups=4, kept=2)[0][0]) == [1]
    # scores as large as 1 each: the higher logit, then the lower id
    assert list(ref.select(np.array([[50.0, 60.0, 60.0, 1.0]]), 3, score="sigmoid")[0][0]) == [1, 2, 0]
    # nothing open
    ids, w, _ = ref.select(np.full((1, 3), -np.inf), 2)
    assert list(ids[0]) == [-1, -1] and not w.any()
    # scores too small for a double, renormalised all the same
    _, w, _ = ref.select(np.array([[-2000.0, -2000.0 + np.log(3), -3000.0]]), 2, score="sigmoid")
    assert w[0] == pytest.approx([0.75, 0.25])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("seed", range(3))
def test_reference_gradient_against_differences(score, renorm, seed):
    rng = np.random.default_rng(seed)
    T, E, k = 3, 7, 4
    z = rng.normal(0, 1.5, (T, E))
    ids = np.argsort(-z, axis=1)[:, :k]
    ids[1, 2] = ids[1, 0]  # an expert picked twice
    ids[2, 1] = -1
    dw = rng.normal(0, 1, (T, k))
    dz, size = ref.select_grad(z, ids, dw, score, renorm, 1.7)
    assert np.all(np.abs(dz) <= size + 1e-15)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = sum(float((dw * ref.select(v, k, score, ids_in=ids, renorm=renorm, scale=1.7)[1]).sum()) * f
                    for v, f in ((up, 1), (dn, -1))) / (2 * h)
            # central differences: truncation h^2 times third derivatives below 50, rounding 2^-52 * 30 / h
            assert abs(dz[t, e] - d) < 1e-8


def test_reference_bias_balance_by_hand():
    bias = np.array([[0.0, 0.5, -np.inf, 0.25, 0.125]], np.float32)
    out = ref.bias_balance(np.array([[4, 1, 90, 1, 2]]), bias, 0.5)
    assert list(out[0]) == [-0.5, 1.0, -np.inf, 0.75, 0.125]  # 8 picks of four open experts: 2 each


def test_reference_lora_by_loops():
    rng = np.random.default_rng(0)
    T, K, N, n, r = 5, 8, 3, 2, 8
    x, a, b = rng.normal(size=(T, K)), rng.normal(size=(n, r, K)), rng.normal(size=(n, N, r))
    ids, ranks, scale, base = np.array([1, 0, -1, 2, 1]), np.array([3, 99]), np.array([2.0, -1.0]), rng.normal(size=(T, N))
    y, size = ref.lora(x, a, b, ids, ranks, scale, base)
    for t in range(T):
        for o in range(N):
            want = base[t, o]
            if ids[t] in (0, 1):
                for j in range(3 if ids[t] == 0 else 8):
                    for i in range(K):
                        want += scale[ids[t]] * b[ids[t], o, j] * a[ids[t], j, i] * x[t, i]
            assert y[t, o] == pytest.approx(want) and abs(y[t, o]) <= size[t, o] + 1e-12


def test_adapters_off_the_gpu_refuse_to_add(mlib):
    torch = pytest.importorskip("torch")
    with pytest.raises(AssertionError, match="on cpu"):
        _pool().add(torch.zeros(2, 64, dtype=torch.bfloat16), 2, torch.zeros(2, dtype=torch.int32), torch.zeros(2, 8))


class _Launched(Exception):
    pass


def _balanced(mlib, monkeypatch):
    """A layer behind a step and its balance(), on the CPU; the launch itself says that it was reached."""
    import contextlib

    import torch

    from expert_vram_slot_amd import layer as layer_py

    def launch(*a):
        raise _Launched
    monkeypatch.setattr(layer_py, "moe_bias_balance", launch)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: 0)
    L = _layer_after_a_step(2, mlib)
    L.stats_out = dict(counts=torch.zeros(8, dtype=torch.int32))
    L.step_layer = L.bound
    L.balanced, L.balanced_layer = (L.steps, 2), L.step_layer
    return L


def test_layer_balance_bias_takes_the_last_steps_counts_alone(mlib, monkeypatch):
    pytest.importorskip("torch")
    L = _balanced(mlib, monkeypatch)
    with pytest.raises(_Launched):
        L.balance_bias(0.001)
    L.steps += 1  # another step, whose counts nobody took
    with pytest.raises(AssertionError, match="last step"):
        L.balance_bias(0.001)
    L.captured = True  # replayed steps are not counted
    with pytest.raises(_Launched):
        L.balance_bias(0.001)


def test_stack_moves_no_bias_by_another_layers_counts(mlib, monkeypatch):
    """Layers of a SlotStack share one SlotLayer: bound anew, its counts are still the last layer's."""
    torch = pytest.importorskip("torch")
    from expert_vram_slot_amd.layer import SlotStack
    stack = SlotStack.__new__(SlotStack)
    stack.layer = L = _balanced(mlib, monkeypatch)
    spec = dict(host_store=None, slot_store=None, G=None)
    stack.layers = [dict(spec, bias=torch.zeros(8)) for _ in range(3)]
    stack.states = [(None,)] * 3
    for l in (0, 2, 0):
        stack.bind(l)
        if l == 0:
            with pytest.raises(_Launched):
                L.balance_bias(0.001)
        else:
            with pytest.raises(AssertionError, match="layer 0's, the bias is layer 2's"):
                L.balance_bias(0.001)
