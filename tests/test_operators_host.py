"""moe_linear_q4, moe_sample and moe_balance_loss without a GPU: refusals and
workspace sizes (nothing is launched on those paths), and the references of
the GPU tests against brute force, closed forms and differences."""
import ctypes

import numpy as np
import pytest

import ops_reference as ref
import synth


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

LINEAR = dict(x=16, x_dtype=1, ldx=64, wq=16, scales=16, group=32, bias=None, T=4, N=8, K=64, y=16, y_dtype=0, ldy=8)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), "ARG"), (dict(wq=None), "ARG"), (dict(scales=None), "ARG"), (dict(y=None), "ARG"),
    (dict(T=-1), "ARG"), (dict(N=0), "ARG"), (dict(K=0), "ARG"), (dict(ldx=63), "ARG"), (dict(ldy=7), "ARG"),
    (dict(ldx=-64), "ARG"),
    (dict(x_dtype=2), "DTYPE"), (dict(y_dtype=-1), "DTYPE"),
    (dict(group=16), "SHAPE"), (dict(group=0), "SHAPE"), (dict(group=48), "SHAPE"), (dict(K=48, ldx=48), "SHAPE"),
    (dict(K=96, ldx=96, group=64), "SHAPE"), (dict(T=(1 << 20) + 1), "SHAPE"), (dict(N=(1 << 22) + 1, ldy=1 << 23), "SHAPE"),
    (dict(ldx=1 << 41), "SHAPE"), (dict(ldy=1 << 41), "SHAPE"),
    (dict(x=24), "ALIGN"), (dict(wq=8), "ALIGN"), (dict(ldx=68), "ALIGN"), (dict(scales=17), "ALIGN"),
    (dict(bias=18), "ALIGN"), (dict(y=18), "ALIGN"), (dict(y=17, y_dtype=1), "ALIGN"),
])
def test_linear_q4_refuses(mlib, change, code):
    a = dict(LINEAR, **change)
    rc = mlib.lib().moe_linear_q4(*[a[n] for n in LINEAR], None)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_linear_q4:")


def test_linear_q4_of_no_tokens(mlib):
    a = dict(LINEAR, T=0, x=None, y=None)
    assert mlib.lib().moe_linear_q4(*[a[n] for n in LINEAR], None) == mlib.MOE_OK


SAMPLE = dict(logits=16, l_dtype=0, ldl=100, T=4, V=100, temperature=None, min_p=None, top_k=None, top_p=None, u=16,
              ids=16, prob=None, ws=16, ws_bytes=1 << 30)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), "ARG"), (dict(u=None), "ARG"), (dict(ids=None), "ARG"), (dict(ws=None), "ARG"),
    (dict(T=-1), "ARG"), (dict(V=0), "ARG"), (dict(ldl=99), "ARG"), (dict(ws_bytes=0), "ARG"),
    (dict(l_dtype=3), "DTYPE"), (dict(T=65536), "SHAPE"), (dict(V=(1 << 20) + 1, ldl=1 << 21), "SHAPE"),
    (dict(logits=18), "ALIGN"), (dict(logits=17, l_dtype=1), "ALIGN"), (dict(ws=8), "ALIGN"),
])
def test_sample_refuses(mlib, change, code):
    a = dict(SAMPLE, **change)
    rc = mlib.lib().moe_sample(*[a[n] for n in SAMPLE], None)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_sample:")


def test_sample_of_no_rows_and_workspace(mlib):
    a = dict(SAMPLE, T=0, logits=None, u=None, ids=None, ws=None, ws_bytes=1 << 30)
    assert mlib.lib().moe_sample(*[a[n] for n in SAMPLE], None) == mlib.MOE_OK
    assert mlib.moe_sample_workspace_bytes(1, 1) > 0
    assert mlib.moe_sample_workspace_bytes(64, 131072) >= mlib.moe_sample_workspace_bytes(1, 131072)
    assert mlib.moe_sample_workspace_bytes(1, 0) == mlib.moe_sample_workspace_bytes(70000, 5) == 0


BALANCE = dict(z=16, z_dtype=0, ids=16, mask=None, T=4, E=8, k=2, counts=16, totals=16, share=16, lse=16, loss=16,
               ws=16, ws_bytes=1 << 30)


@pytest.mark.parametrize("change,code", [
    (dict(z=None), "ARG"), (dict(ids=None), "ARG"), (dict(counts=None), "ARG"), (dict(totals=None), "ARG"),
    (dict(share=None), "ARG"), (dict(lse=None), "ARG"), (dict(loss=None), "ARG"), (dict(ws=None), "ARG"),
    (dict(T=-1), "ARG"), (dict(E=0), "ARG"), (dict(k=0), "ARG"), (dict(ws_bytes=8), "ARG"),
    (dict(z_dtype=5), "DTYPE"), (dict(E=4097), "SHAPE"), (dict(k=9), "SHAPE"), (dict(E=64, k=33), "SHAPE"),
    (dict(T=(1 << 24) + 1), "SHAPE"), (dict(z=20), "ALIGN"), (dict(ws=8), "ALIGN"), (dict(share=20), "ALIGN"),
])
def test_balance_refuses(mlib, change, code):
    a = dict(BALANCE, **change)
    rc = mlib.lib().moe_balance_loss(*[a[n] for n in BALANCE], None)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_balance_loss:")


GRAD = dict(z=16, z_dtype=0, lse=16, mask=None, counts=16, totals=16, dloss=16, T=4, E=8, dz=16)


@pytest.mark.parametrize("change,code", [
    (dict(z=None), "ARG"), (dict(lse=None), "ARG"), (dict(counts=None), "ARG"), (dict(totals=None), "ARG"),
    (dict(dloss=None), "ARG"), (dict(dz=None), "ARG"), (dict(T=-1), "ARG"), (dict(E=0), "ARG"),
    (dict(z_dtype=2), "DTYPE"), (dict(E=4097), "SHAPE"), (dict(T=(1 << 24) + 1), "SHAPE"), (dict(z=20), "ALIGN"),
    (dict(dz=8), "ALIGN"),
])
def test_balance_grad_refuses(mlib, change, code):
    a = dict(GRAD, **change)
    rc = mlib.lib().moe_balance_loss_bwd(*[a[n] for n in GRAD], None)
    assert rc == getattr(mlib, "MOE_E_" + code), mlib.moe_last_error()
    assert mlib.moe_last_error().startswith("moe_balance_loss_bwd:")


def test_balance_workspace(mlib):
    assert mlib.moe_balance_workspace_bytes(0, 1) > 0
    assert mlib.moe_balance_workspace_bytes(4096, 512) >= mlib.moe_balance_workspace_bytes(1, 512)
    assert mlib.moe_balance_workspace_bytes(1, 4097) == mlib.moe_balance_workspace_bytes(-1, 8) == 0


def test_binding_raises_with_the_reason(mlib):
    with pytest.raises(mlib.MoeError) as e:
        mlib.moe_linear_q4(16, 1, 64, 16, 16, 7, None, 1, 8, 64, 16, 0, 8, stream=0)
    assert e.value.code == mlib.MOE_E_SHAPE and "groups of 7" in str(e.value)
    with pytest.raises(mlib.MoeError):
        mlib.moe_sample(None, 0, 8, 1, 8, None, None, None, None, 16, 16, None, 16, 1 << 20, stream=0)
    with pytest.raises(mlib.MoeError):
        mlib.moe_balance_loss(16, 0, 16, None, 1, 8, 9, 16, 16, 16, 16, 16, 16, 1 << 20, stream=0)
    with pytest.raises(mlib.MoeError):
        mlib.moe_balance_loss_bwd(None, 0, 16, None, 16, 16, 16, 1, 8, 16, stream=0)


# ------------------------------------------------------------ references


@pytest.mark.parametrize("change", [dict(V=9), dict(H=128), dict(group=128), dict(bias="short"), dict(scales="f32"),
                                    dict(wq="strided")])
def test_decode_head_refuses(mlib, change):
    torch = pytest.importorskip("torch")
    from expert_vram_slot_amd.layer import DecodeHead
    a = dict(H=64, V=8, wq=torch.zeros(8, 32, dtype=torch.uint8), scales=torch.zeros(8, 2, dtype=torch.float16), group=32,
             T_max=2, device="cpu")
    DecodeHead(**a)
    change = dict(change)
    if "bias" in change:
        change["bias"] = torch.zeros(7)
    if "scales" in change:
        change["scales"] = torch.zeros(8, 2)
    if "wq" in change:
        change["wq"] = torch.zeros(8, 64, dtype=torch.uint8)[:, ::2]
    with pytest.raises(AssertionError):
        DecodeHead(**{**a, **change})


@pytest.mark.parametrize("change", [
    dict(x="f32"), dict(x="f16"), dict(x="short"), dict(x="few rows"), dict(x="every other column"), dict(x="numpy"),
    dict(x="elsewhere"), dict(T=3), dict(u="f64"), dict(u="short"), dict(u="strided"), dict(u="elsewhere"),
    dict(temperature="f64"), dict(min_p="f16"), dict(top_p="short"), dict(top_k="i64"), dict(top_k="f32"),
    dict(top_k="short"), dict(u=None)])
def test_decode_head_step_refuses(change):
    """What the kernels would read as something else, or past its end (nothing is launched: the head is on the CPU)."""
    torch = pytest.importorskip("torch")
    from expert_vram_slot_amd.layer import DecodeHead
    head = DecodeHead(H=64, V=8, wq=torch.zeros(8, 32, dtype=torch.uint8), scales=torch.zeros(8, 2, dtype=torch.float16),
                      group=32, T_max=2, device="cpu")
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    bad = {"f32": torch.zeros(2), "f64": torch.zeros(2, dtype=torch.float64), "f16": torch.zeros(2, dtype=torch.float16),
           "i64": torch.zeros(2, dtype=torch.int64), "short": torch.zeros(1), "strided": torch.zeros(4)[::2],
           "elsewhere": torch.zeros(2, device="meta"), None: None}
    bad_x = {"f32": x.float(), "f16": x.half(), "short": x.reshape(-1)[:127], "few rows": x[:1],
             "every other column": torch.zeros(2, 128, dtype=torch.bfloat16)[:, ::2], "numpy": x.float().numpy(),
             "elsewhere": torch.zeros(2, 64, dtype=torch.bfloat16, device="meta")}
    a = dict(x=x, T=2, u=torch.zeros(2))
    for name, value in change.items():
        a[name] = value if name == "T" else bad_x[value] if name == "x" else bad[value]
        if (name, value) == ("top_k", "short"):
            a[name] = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(AssertionError):
        head.step(**a)


@pytest.mark.parametrize("what", ["wq", "scales", "bias", "strided bias"])
def test_decode_head_refuses_weights_elsewhere(what):
    torch = pytest.importorskip("torch")
    from expert_vram_slot_amd.layer import DecodeHead
    a = dict(H=64, V=8, wq=torch.zeros(8, 32, dtype=torch.uint8), scales=torch.zeros(8, 2, dtype=torch.float16), group=32,
             T_max=2, device="cpu", bias=torch.zeros(8))
    DecodeHead(**a)
    a.update({"bias": torch.zeros(16)[::2]} if what == "strided bias" else {what: a[what].to("meta")})
    with pytest.raises(AssertionError):
        DecodeHead(**a)


def _layer_after_a_step(T):
    """The part of a SlotLayer that balance() looks at, on the CPU, as a step of T tokens leaves it."""
    import torch

    from expert_vram_slot_amd.layer import SlotLayer
    L = SlotLayer.__new__(SlotLayer)
    L.E, L.k, L.T_max, L.stats_out = 8, 2, 4, None
    L.logits, L.ids = torch.zeros(32), torch.zeros(8, dtype=torch.int32)
    L.steps, L.step_T, L.captured, L.balanced = 1, T, False, None
    return L


@pytest.mark.parametrize("change", [dict(T=3), dict(T=5), dict(mask="i64"), dict(mask="f32"), dict(mask="short"),
                                    dict(mask="strided"), dict(mask="elsewhere"), dict(mask="numpy")])
def test_layer_balance_refuses(change):
    torch = pytest.importorskip("torch")
    L = _layer_after_a_step(2)
    bad = {"i64": torch.ones(2, dtype=torch.int64), "f32": torch.ones(2), "short": torch.ones(1, dtype=torch.uint8),
           "strided": torch.ones(4, dtype=torch.uint8)[::2], "elsewhere": torch.ones(2, dtype=torch.uint8, device="meta"),
           "numpy": np.ones(2, np.uint8)}
    a = dict(T=2)
    a.update((n, bad.get(v, v)) for n, v in change.items())
    with pytest.raises(AssertionError):
        L.balance(**a)


@pytest.mark.parametrize("change", [dict(T=1), dict(mask="i64"), dict(mask="short"), dict(dloss="f64"), dict(dloss="short"),
                                    dict(dloss="strided"), dict(dloss="elsewhere"), dict(dloss=(1.0, 0.1)),
                                    dict(before="no balance"), dict(before="another step")])
def test_layer_balance_grad_refuses(change):
    torch = pytest.importorskip("torch")
    L = _layer_after_a_step(2)
    L.stats_out, L.balanced = dict(lse=torch.zeros(4), counts=torch.zeros(8), totals=torch.zeros(2)), (1, 2)
    bad = {"i64": torch.ones(2, dtype=torch.int64), "short": torch.ones(1), "f64": torch.ones(2, dtype=torch.float64),
           "strided": torch.ones(4)[::2], "elsewhere": torch.ones(2, device="meta")}
    a = dict(T=2, dloss=torch.ones(2))
    for n, v in change.items():
        if v == "no balance":
            L.stats_out = L.balanced = None
        elif v == "another step":
            L.steps += 1
        elif (n, v) == ("mask", "short"):
            a[n] = torch.ones(1, dtype=torch.uint8)
        else:
            a[n] = bad.get(v, v) if isinstance(v, str) else v
    with pytest.raises(AssertionError):
        L.balance_grad(**a)


def test_reference_codes_are_the_slab_planes():
    """The nibble order is a Q4B32 slab's: decoding the generator's gate plane gives the oracle's weights."""
    import oracle
    H, I = 64, 32
    rng = np.random.default_rng(0)
    w = [rng.normal(0, 1, s).astype(np.float32) for s in ((I, H), (I, H), (H, I))]
    slab = synth.encode_slab(synth.W_Q4B32, H, I, *w)
    wq = slab[:I * H // 2].reshape(I, H // 2)
    d = slab[I * H // 2:I * H // 2 + I * H // 16].view(np.float16).reshape(I, H // 32)
    got = (ref.codes(wq).astype(np.float64) - 8) * np.repeat(d.astype(np.float64), 32, axis=1)
    want = oracle.decode_expert(synth.W_Q4B32, slab, H, I)[0]
    np.testing.assert_array_equal(got, np.asarray(want, np.float64).reshape(I, H))


def test_reference_sample_hand_cases():
    l = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    # masses 1 4 2 1 of 8, ascending ids: 0 [0, 1/8), 1 [1/8, 5/8), 2 [5/8, 7/8), 3 [7/8, 1)
    for u, want, prob in ((0.0, 0, .125), (0.124, 0, .125), (0.2, 1, .5), (0.7, 2, .25), (0.9, 3, .125), (1.0, 3, .125)):
        assert ref.sample_row(l, u)[:2] == pytest.approx((want, prob))
    assert list(ref.sample_row(l, 0.5, top_k=2)[2]) == [1, 2]
    assert list(ref.sample_row(l, 0.5, top_k=3)[2]) == [0, 1, 2]  # of two equal logits the lower id
    assert list(ref.sample_row(l, 0.5, top_p=0.49)[2]) == [1]
    assert list(ref.sample_row(l, 0.5, top_p=0.51)[2]) == [1, 2]
    assert list(ref.sample_row(l, 0.5, min_p=0.3)[2]) == [1, 2]
    assert list(ref.sample_row(l, 0.5, top_k=2, top_p=0.66)[2]) == [1]  # 4 of the 6 that top-k left
    assert ref.sample_row(l, 0.9, temperature=0.0)[:2] == (1, 1.0)
    assert ref.sample_row(np.full(3, -np.inf), 0.5)[0] == -1
    # temperature 1/2 squares the masses: 1 16 4 1 of 22
    assert ref.sample_row(l, 0.5, temperature=0.5)[1] == pytest.approx(16 / 22)


@pytest.mark.parametrize("seed", range(20))
def test_reference_sample_against_brute_force(seed):
    """Each cut against its definition over every prefix of a small row."""
    rng = np.random.default_rng(seed)
    V = int(rng.integers(1, 9))
    l = rng.integers(-3, 4, V).astype(np.float64)  # ties are common
    temperature, min_p = float(rng.uniform(0.5, 2)), float(rng.choice([0, 0.05, 0.3]))
    top_k, top_p, u = int(rng.integers(0, V + 2)), float(rng.uniform(0, 1.1)), float(rng.uniform())
    order = sorted(range(V), key=lambda i: (-l[i], i))
    w = {i: np.exp((l[i] - l.max()) / temperature) for i in range(V)}
    left = [i for i in order if w[i] >= min_p]
    if top_k > 0:
        left = left[:top_k]
    if top_p < 1:
        total = sum(w[i] for i in left)
        left = next(left[:n] for n in range(1, len(left) + 1) if sum(w[i] for i in left[:n]) >= top_p * total * (1 - 1e-15))
    got, prob, kept = ref.sample_row(l, u, temperature, min_p, top_k, top_p)
    assert sorted(left) == list(kept)
    total, run = sum(w[i] for i in left), 0.0
    for i in sorted(left):
        run += w[i]
        if run > u * total:
            break
    assert got == i and prob == pytest.approx(w[i] / total)


def test_reference_balance_closed_forms():
    # uniform logits and even picks: loss 1; every pick and all mass on one expert: loss E
    z, ids = np.zeros((8, 4)), np.arange(8, dtype=np.int32).reshape(8, 1) % 4
    o = ref.balance(z, ids)
    assert o["loss"][0] == pytest.approx(1.0) and o["loss"][1] == pytest.approx(np.log(4) ** 2)
    np.testing.assert_array_equal(o["counts"], [2, 2, 2, 2])
    z = np.full((3, 4), -np.inf)
    z[:, 2] = 5.0
    o = ref.balance(z, np.full((3, 1), 2, np.int32))
    assert o["loss"][0] == 4.0 and o["loss"][1] == 25.0
    np.testing.assert_array_equal(o["share"], [0, 0, 1, 0])


@pytest.mark.parametrize("seed", range(4))
def test_reference_balance_gradient_against_differences(seed):
    rng = np.random.default_rng(seed)
    T, E, k = 5, 6, 2
    z = rng.normal(0, 1.5, (T, E))
    ids = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    mask = np.array([1, 0, 1, 1, 1], np.uint8) if seed % 2 else None
    dloss = np.array([0.7, -0.3])
    g = ref.balance_grad(z, ids, dloss, mask)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = dloss @ (ref.balance(up, ids, mask)["loss"] - ref.balance(dn, ids, mask)["loss"]) / (2 * h)
            # central differences: truncation h^2 (1e-12), rounding 2^-52 * loss / h (loss below 50)
            assert abs(g[t, e] - d) < 2e-8
