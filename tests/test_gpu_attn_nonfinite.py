"""Attention of rows that meet NaN, infinity or scores past fp32's range: such a
row is NaN and so is its lse, however the call is cut into parts, and the rows
beside it are as if nothing had been there."""

import math

import pytest
import torch

import attn_ref as R
from test_gpu_attn_tree import TYPES, _call, _make

pytestmark = pytest.mark.gpu

# the parts that the keys are cut into for the sequences below, and the pages
# of a table row: one, few parts (joined by a wave a row), many (by four)
WIDTHS = {1: 27, 8: 128, 40: 640}


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


def _rows(q, k, v, scale, seen, dtype):
    """Checks of one head's rows: q [R,dk], k [L,dk], v [L,dv], seen [R,L] in
    64 bits.  Returns check(out [R,dv], lse [R], gate logits or None)."""
    # the scores in fp32's range: what overflows there is infinite
    s = ((q @ k.T) * scale).float().double()
    some = seen.any(1)
    finite = seen & torch.isfinite(s)
    # a key that is infinitely far has no weight beside one that is not
    good = some & (finite | torch.isneginf(s) | ~seen).all(1) & finite.any(1)
    odd = (seen[:, :, None] & ~torch.isfinite(v)[None]).any(1)  # [R, dv]

    def check(name, out, lse, z=None):
        out, lse = out.double(), lse.double()
        assert bool((out[~some] == 0).all()) and bool(torch.isneginf(lse[~some]).all()), name
        broken = some & ~good
        assert bool(torch.isnan(out[broken]).all()), (name, "out", out[broken])
        assert bool(torch.isnan(lse[broken]).all()), (name, "lse", lse[broken])
        if not bool(good.any()):
            return
        clean = torch.where(torch.isfinite(k).all(1, keepdim=True), k, torch.zeros_like(k))
        o, bo, l, bl, _, _ = R.softmax_rows(q[good], clean, v, scale, finite[good], R.UNIT[dtype])
        if z is not None:
            g = torch.sigmoid(z[good].double())
            o, bo = o * g, bo * g + o.abs() * g * 2.0 ** -20
        bo = bo + R.UNIT[dtype] * (o.abs() + bo) + 1e-30
        assert not bool(torch.isfinite(out[good][odd[good]]).any()), (name, "values")
        fine = ~odd[good]
        R.check(name + " out", out[good][fine], o[fine], bo[fine])
        R.check(name + " lse", lse[good], l, bl)
    return check


def _check_tree(K, x, dtype):
    out, lse = _call(K, x)
    B, T, H, dk = x["q"].shape
    G = H // x["k_new"].shape[2]
    for b in range(B):
        n = x["ctx_k"][b].shape[0]
        new = torch.tensor([[bool(int(x["mask"][b, t]) >> j & 1) for j in range(T)] for t in range(T)], device="cuda")
        seen = torch.cat([torch.ones(T, n, dtype=torch.bool, device="cuda"), new], 1)
        for h in range(H):
            k = torch.cat([x["ctx_k"][b][:, h // G], x["k_new"][b, :, h // G]]).double()
            v = torch.cat([x["ctx_v"][b][:, h // G], x["v_new"][b, :, h // G]]).double()
            z = None if x["z"] is None else x["z"][b, :, h]
            _rows(x["q"][b, :, h].double(), k, v, dk ** -0.5, seen, dtype)(f"{b},{h}", out[b, :, h], lse[b, :, h], z)
    return out, lse


def _tree(K, parts, dtype, dk=64, dv=64, lens=(300, 40), T=5):
    x = _make(31, list(lens), T, 4, 2, dk, dv, 16, TYPES[dtype], gate=True, width=WIDTHS[parts])
    need = K.kda_attn_tree_workspace_bytes(len(lens), T, 4, 2, dk, dv, TYPES[dtype], WIDTHS[parts] * 16)
    each = len(lens) * T * 4 * (dv * 4 + 8)
    assert (need == 0) if parts == 1 else parts * each <= need < (parts + 1) * each, "not cut as the test means it"
    return x


def _committed(x, b, token, head, **to):
    """Overwrites a committed token's key or value, in the cache and beside it."""
    page = int(x["table"][int(x["rows"][b]), token // 16])
    for name, pool, ctx in (("k", "kc", "ctx_k"), ("v", "vc", "ctx_v")):
        if name in to:
            for ch, value in to[name].items():
                x[pool][page, head, token % 16, ch] = value
                x[ctx][b][token, head, ch] = value


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("parts", WIDTHS)
class TestTree:
    def test_a_query(self, K, parts, dtype):
        x = _tree(K, parts, dtype)
        x["q"][0, 1, 2, 5] = math.nan
        x["q"][0, 4, 0, 63] = -math.inf
        x["q"][1, 0, 3, 0] = math.inf
        _check_tree(K, x, TYPES[dtype])

    @pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
    @pytest.mark.parametrize("token", [0, 70, 299])
    def test_a_committed_key(self, K, parts, dtype, token, value):
        """Every row of its head: NaN; an infinite one where the score is +infinity."""
        x = _tree(K, parts, dtype)
        _committed(x, 0, token, 1, k={3: value})
        _check_tree(K, x, TYPES[dtype])

    @pytest.mark.parametrize("value", [math.nan, math.inf])
    def test_a_draft_key(self, K, parts, dtype, value):
        """The rows that attend the draft, and no others."""
        x = _tree(K, parts, dtype)
        x["k_new"][0, 2, 0, 9] = value
        x["k_new"][1, 4, 1, 0] = value
        _check_tree(K, x, TYPES[dtype])

    def test_scores_that_overflow(self, K, parts, dtype):
        """A row whose own scores are past fp32's range is NaN.  The rows beside
        it have scores of 10^29: the largest takes all the weight."""
        x = _tree(K, parts, dtype)
        x["q"][0, 3, 1, 8] = 1e30
        _committed(x, 0, 33, 0, k={8: 1e30})
        _committed(x, 0, 200, 0, k={8: -1e30})
        _check_tree(K, x, TYPES[dtype])

    @pytest.mark.parametrize("value", [math.nan, math.inf])
    def test_a_committed_value(self, K, parts, dtype, value):
        """The channel, also where the weights of the key and of all around it
        are too small for fp32."""
        x = _tree(K, parts, dtype)
        _committed(x, 0, 100, 0, v={7: value})
        x["q"][:, :, :, 0] = 4.0
        for token in range(128, 224):
            _committed(x, 0, token, 1, k={0: -1e4}, v={9: value} if token == 170 else {})
        _check_tree(K, x, TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("parts", WIDTHS)
def test_rows_whose_scores_are_all_minus_infinity(K, parts, dtype):
    """NaN: only a row that attends nothing is 0 with an lse of -infinity."""
    x = _tree(K, parts, dtype, lens=(300, 40, 0))
    x["q"][:, :, :, 0] = 1.5
    for token in range(40):
        _committed(x, 1, token, 1, k={0: -math.inf})
    x["k_new"][2, 1, 0, 0] = -math.inf
    x["mask"][1, 2], x["mask"][2, 3], x["mask"][2, 4] = 0, 1 << 1 | 1 << 40, 1 << 5
    out, lse = _check_tree(K, x, TYPES[dtype])
    assert bool(torch.isnan(out[1, 2, 2:]).all()) and bool(torch.isnan(out[2, 3, :2]).all())
    assert bool((out[2, 4] == 0).all())


@pytest.mark.parametrize("parts", WIDTHS)
def test_other_head_sizes(K, parts):
    for dk, dv in ((16, 16), (32, 32), (128, 128), (192, 128)):
        for dtype in ("f32", "bf16"):
            print(f"not finite {dk}/{dv} {dtype}", flush=True)
            x = _tree(K, parts, dtype, dk, dv)
            x["q"][0, 2, 1, dk - 1] = math.nan
            _committed(x, 1, 17, 1, k={dk - 1: math.nan})
            x["k_new"][0, 1, 1, 4] = math.inf
            _check_tree(K, x, TYPES[dtype])


def _prefill(K, q, k, v, z, dtype):
    """One sequence, every head's rows checked."""
    out, lse = K.kda_attn_prefill(q, k, v, out_gate=z)
    torch.cuda.synchronize()
    n, H, dk = q.shape
    seen, G = R.causal(n, "cuda"), H // k.shape[1]
    for h in range(H):
        _rows(q[:, h].double(), k[:, h // G].double(), v[:, h // G].double(), dk ** -0.5, seen, dtype)(
            f"head {h}", out[:, h], lse[:, h], None if z is None else z[:, h])
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("which", ["query", "key", "far", "overflow"])
def test_prefill(K, which, dk, dv, dtype):
    t = TYPES[dtype]
    g = torch.Generator(device="cuda")
    g.manual_seed(dk)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(t)  # noqa: E731
    q, k, v, z = new(150, 4, dk), new(150, 2, dk), new(150, 2, dv), new(150, 4, dv)
    print(f"prefill {which} {dk}/{dv} {dtype}", flush=True)
    if which == "query":
        q[5, 0, 3], q[70, 1, 0], q[149, 3, dk - 1] = math.nan, math.inf, -math.inf
    elif which == "key":
        k[40, 0, 2], k[100, 1, 1] = math.nan, math.inf
    elif which == "overflow":
        q[120, 2, 4], k[20, 1, 4] = 1e30, 1e30
    else:  # the first rows attend scores of -infinity alone
        q[:, :, 1] = 0.5
        k[:3, 0, 1], k[60, 1, 1] = -math.inf, -math.inf
    out, lse = _prefill(K, q, k, v, z, t)
    # the gradients of a broken row are NaN, and reach what the row attends
    dy = new(150, 4, dv)
    grads = K.kda_attn_prefill_backward(q, k, v, out, lse, dy, out_gate=z)
    torch.cuda.synchronize()
    broken = torch.isnan(lse)
    assert bool(broken.any()) and bool(torch.isnan(grads["dq"][broken]).all())
    for h in range(4):
        if bool(broken[:, h].any()):
            last = int(torch.nonzero(broken[:, h])[-1, 0])
            for name in ("dk", "dv"):
                assert bool(torch.isnan(grads[name][:last + 1, h // 2]).all()), name


FAR = 1024.0  # its square is every score's size below; the scores are whole numbers, exact in fp32


def _check_far(name, out, lse, q, k, v, seen, dtype):
    """Scores of FAR^2 and a small number: the weights are those of the small
    numbers alone, and lse is FAR^2 more (three roundings of a 24-bit number)."""
    q, k = q.double().clone(), k.double().clone()
    assert bool((q[:, 0] * k[:, 0].unique() == FAR * FAR).all())
    q[:, 0] = 0
    o, bo, l, bl, _, _ = R.softmax_rows(q, k, v.double(), 1.0, seen, R.UNIT[dtype])
    R.check(name + " out", out, o, bo + R.UNIT[dtype] * (o.abs() + bo) + 1e-30)
    R.check(name + " lse", lse, l + FAR * FAR, bl + 3 * FAR * FAR * 2.0 ** -24)


def _far_row(q):
    q.zero_()
    q[..., 0], q[..., 1] = FAR, 1.0


def _far_key(k):
    k[..., 0], k[..., 1] = FAR, k[..., 1].round()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("parts", WIDTHS)
def test_large_scores_keep_their_differences(K, parts, dtype):
    t = TYPES[dtype]
    x = _tree(K, parts, dtype)
    x["z"] = None
    _far_row(x["q"])
    for y in (x["kc"], x["k_new"], *x["ctx_k"]):
        _far_key(y)
    out, lse = _call(K, x, scale=1.0)
    for b in range(2):
        new = torch.tensor([[bool(int(x["mask"][b, i]) >> j & 1) for j in range(5)] for i in range(5)], device="cuda")
        seen = torch.cat([torch.ones(5, x["ctx_k"][b].shape[0], dtype=torch.bool, device="cuda"), new], 1)
        for h in range(4):
            _check_far(f"{b},{h}", out[b, :, h], lse[b, :, h], x["q"][b, :, h], torch.cat([x["ctx_k"][b][:, h // 2], x["k_new"][b, :, h // 2]]),
                       torch.cat([x["ctx_v"][b][:, h // 2], x["v_new"][b, :, h // 2]]), seen, t)
    g = torch.Generator(device="cuda")
    g.manual_seed(parts)
    q, k, v = (torch.randn(n, generator=g, device="cuda").to(t) for n in ((200, 2, 128), (200, 1, 128), (200, 1, 128)))
    _far_row(q)
    _far_key(k)
    out, lse = K.kda_attn_prefill(q, k, v, scale=1.0)
    for h in range(2):
        _check_far(f"prefill {h}", out[:, h], lse[:, h], q[:, h], k[:, 0], v[:, 0], R.causal(200, "cuda"), t)
