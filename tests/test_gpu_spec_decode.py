"""GPU parity of the speculative decoding calls against the fp64 oracle (oracle/spec_oracle.py), through the C ABI.

Tolerances are derived, not tuned:
  * kvq_qk_norm_rope: one bf16 rounding (2^-8 of the value) of an fp32 result; norm and rotation are fewer than
    16 fp32 operations on values of at most |a| + |b| (2^-20), the fixed-point angle is off by at most 2^-30 turns
    in 2^31 steps plus the 2^-50 relative error of the frequency times the position;
  * kvq_decode_attention_tree: the oracle's `slack` (f16 operands), plus one bf16 rounding for bf16 outputs;
  * kvq_verify_tree: equal;  kvq_append_accepted: equal, bit for bit.
"""
import math
import zlib

import numpy as np
import pytest

from oracle import kvq_oracle as O
from oracle import spec_oracle as S
from quantized_kv_cache_decode_gb300 import inputs as I

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kvq_testlib as TL  # noqa: E402
from quantized_kv_cache_decode_gb300 import kvq  # noqa: E402

F32 = np.float32


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def bf16_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).astype(np.int16)).cuda().view(torch.bfloat16)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().astype(np.uint16)


# --------------------------------------------------------------------------- #
# norm and rotation
# --------------------------------------------------------------------------- #

ROPE = [
    # batch, tokens, q heads, kv heads, base, rotate keys, q norm, k norm, pad, eps
    (1, 1, 1, 1, 10000.0, True, True, True, 0, 1e-6),
    (16, 1, 32, 8, 500000.0, True, True, True, 0, 1e-5),
    (3, 7, 5, 5, 10000.0, False, True, False, 8, 1e-6),
    (2, 33, 48, 8, 500000.0, True, False, True, 64, 0.0),
    (2, 5, 8, 1, 0.0, True, True, True, 0, 1e-6),
    (1, 700, 12, 2, 1.0001, True, False, False, 200, 1e-6),
    (5, 131, 64, 8, 10000.0, True, True, True, 0, 1e-6),
]


@pytest.mark.parametrize("case", ROPE, ids=[f"B{c[0]}n{c[1]}q{c[2]}k{c[3]}base{c[4]:g}" for c in ROPE])
def test_qk_norm_rope(case):
    B, n, hq, h, base, rotk, qn, kn, pad, eps = case
    rng = np.random.default_rng(zlib.crc32(repr(case).encode()))
    stride = (hq + 2 * h) * 128 + pad
    x = rng.standard_normal((B * n, stride)).astype(F32) * np.exp2(rng.integers(-6, 7, (B * n, 1))).astype(F32)
    xb = I.f32_to_bf16_bits(x)
    w = [I.f32_to_bf16_bits((1 + 0.3 * rng.standard_normal(128)).astype(F32)) for _ in range(2)]
    pos = rng.integers(-100, 200000, (B, n)).astype(np.int32)
    pos.reshape(-1)[:3] = [2 ** 31 - 1, -2 ** 31, 0][:min(3, B * n)]
    rows, pd = bf16_dev(xb), dev(pos)
    wd = [bf16_dev(a) for a in w]
    q = torch.full((B, n, hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.full((B, h, n, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kvq.qk_norm_rope(rows, stride, B, n, hq, h, wd[0] if qn else None, wd[1] if kn else None, eps,
                     pd if base else None, base, rotk, q, k, v)
    torch.cuda.synchronize()
    xf = I.bf16_bits_to_f32(xb)[:, :(hq + 2 * h) * 128].reshape(B * n, hq + 2 * h, 128)
    wf = [I.bf16_bits_to_f32(a) for a in w]
    p = pos.reshape(-1)
    assert np.array_equal(bits_of(v).transpose(0, 2, 1, 3).reshape(B * n, h, 128),
                          xb[:, :(hq + 2 * h) * 128].reshape(B * n, hq + 2 * h, 128)[:, hq + h:])
    got_q = q.float().cpu().numpy().reshape(B * n, hq, 128)
    got_k = k.float().cpu().numpy().transpose(0, 2, 1, 3).reshape(B * n, h, 128)
    for got, src, wt, normed, turn in ((got_q, xf[:, :hq], wf[0], qn, base > 0),
                                       (got_k, xf[:, hq:hq + h], wf[1], kn, base > 0 and rotk)):
        for i in range(src.shape[1]):
            y = S.head_norm(src[:, i], wt if normed else None, eps)
            ref = S.rotate_exact(y, p, float(F32(base))) if turn else y  # (the call takes an fp32 base)
            mag = np.abs(y) + np.abs(np.roll(y, 64, -1))
            ang = (2.0 ** -29 + np.abs(p.astype(np.float64)) * 2.0 ** -49)[:, None]
            tol = 2.0 ** -8 * np.abs(ref) + mag * (2.0 ** -20 + ang)
            worst = float((np.abs(got[:, i] - ref) - tol).max())
            assert worst <= 0, (i, worst)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_qk_norm_rope_heads_whose_squares_leave_fp32(eps):
    # values of 2^-130 to 2^126 next to ordinary ones in one warp: the formula's result, not 0 or infinity
    hq, h, n = 6, 2, 40
    rng = np.random.default_rng(3)
    x = rng.standard_normal((n, hq + 2 * h, 128)).clip(-3, 3)
    e = rng.choice([-130, -100, -60, -45, 0, 45, 64, 90, 126], (n, hq + 2 * h, 1))
    xb = I.f32_to_bf16_bits((x * np.exp2(e.astype(np.float64)) * 0.5).astype(F32))
    w = [I.f32_to_bf16_bits((1 + 0.3 * rng.standard_normal(128)).astype(F32)) for _ in range(2)]
    pos = rng.integers(0, 5000, (1, n)).astype(np.int32)
    q = torch.empty(1, n, hq, 128, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(1, h, n, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kvq.qk_norm_rope(bf16_dev(xb), (hq + 2 * h) * 128, 1, n, hq, h, *(bf16_dev(a) for a in w), eps, dev(pos), 1e4, True,
                     q, k, v)
    torch.cuda.synchronize()
    xf = I.bf16_bits_to_f32(xb)
    got = np.concatenate([q.double().cpu().numpy()[0], k.double().cpu().numpy()[0].transpose(1, 0, 2)], 1)
    for i in range(hq + h):
        y = S.head_norm(xf[:, i], I.bf16_bits_to_f32(w[i >= hq]), float(F32(eps)))
        ref = S.rotate_exact(y, pos[0], 1e4)
        mag = np.abs(y) + np.abs(np.roll(y, 64, -1))
        # (half a step of a bf16 subnormal is 2^-134: outputs may be that small beside an eps)
        tol = 2.0 ** -8 * np.abs(ref) + mag * (2.0 ** -20 + 2.0 ** -29 + 5000 * 2.0 ** -49) + 2.0 ** -134
        assert (np.abs(got[:, i] - ref) <= tol).all(), (i, float((np.abs(got[:, i] - ref) / tol).max()))
    assert np.array_equal(bits_of(v)[0].transpose(1, 0, 2), xb[:, hq + h:])


def test_tree_workspace_of_the_largest_batch():
    for fmt, G, Gv, R, kw in (("int8", 16, 16, 32, {}), ("int4", 32, 128, 32, {}), ("int2", 16, 16, 0, {}),
                              ("fp8_e4m3", 1, 128, 0, {}), ("bf16", 0, 0, 0, {}), ("int8", 256, 16, 256, {})):
        cfg = kvq.make_config(fmt, 1, G, Gv, R, 0, capacity_tokens=1024, **kw)
        for n, hq in ((1, 1), (8, 8), (64, 8)):
            assert kvq.decode_workspace_size_tree(cfg, 2048, n, hq) > 0, (fmt, n, hq)


# --------------------------------------------------------------------------- #
# tree attention
# --------------------------------------------------------------------------- #


def build(fmt, H, lens, G, Gv, R, S_, paged, seed, block_tokens=16, scale=10.0, extra=0):
    """A GPU cache of `lens` tokens and its oracle twins (as in test_gpu_parity)."""
    gl = TL.GpuLayer(fmt, H, lens, G, Gv, R, S_, paged=paged, block_tokens=block_tokens, seed=seed,
                     extra_capacity=extra)
    rng = np.random.default_rng(seed)
    mask = np.zeros(128, bool)
    mask[rng.choice(128, 4, replace=False)] = True
    kv = {(b, h): (I.random_bf16(seed * 1000 + 2 * (b * H + h), (T, 128), outlier_mask=mask, outlier_scale=scale),
                   I.random_bf16(seed * 1000 + 2 * (b * H + h) + 1, (T, 128)))
          for b, T in enumerate(lens) for h in range(H)}
    ks = vs = None
    if gl.fp8:
        ka = np.concatenate([kv[i][0].reshape(-1) for i in kv] + [I.f32_to_bf16_bits(np.array([30.0], F32))])
        va = np.concatenate([kv[i][1].reshape(-1) for i in kv] + [I.f32_to_bf16_bits(np.array([4.5], F32))])
        gl.calibrate_fp8(ka, va)
        ks, vs = O.fp8_tensor_scale(O.bf16_to_f32(ka), fmt), O.fp8_tensor_scale(O.bf16_to_f32(va), fmt)
    for b, T in enumerate(lens):
        if T:
            gl.append(b, np.stack([kv[b, h][0] for h in range(H)]), np.stack([kv[b, h][1] for h in range(H)]), 0)
    torch.cuda.synchronize()
    caches = [[O.build_head_cache(O.bf16_to_f32(kv[b, h][0]), O.bf16_to_f32(kv[b, h][1]), gl.spec, ks, vs)
               for h in range(H)] for b in range(len(lens))]
    return gl, caches


def random_tree(rng, n, kind):
    if kind == "chain":
        return np.arange(n) - 1
    if kind == "star":
        return np.where(np.arange(n) > 0, 0, -1)
    if kind == "roots":
        return np.full(n, -1)
    return np.array([-1 if i == 0 or rng.random() < 0.1 else rng.integers(max(0, i - 5), i) for i in range(n)])


def draft_inputs(seed, B, H, g, N):
    q = I.random_bf16(seed + 1, (B, N, H * g, 128))
    mask = np.zeros(128, bool)
    mask[::41] = True
    k = I.random_bf16(seed + 2, (B, H, N, 128), outlier_mask=mask, outlier_scale=6.0)
    v = I.random_bf16(seed + 3, (B, H, N, 128))
    return q, k, v


def tree_call(gl, q, k, v, parents, out_bf16=False, lens=None, want_lse=True, scale=None, ws=None, stream=None):
    B, N, Hq = q.shape[:3]
    out = torch.full((B, N, Hq, 128), float("nan"), dtype=torch.bfloat16 if out_bf16 else torch.float32, device="cuda")
    lse = torch.full((B, N, Hq), float("nan"), dtype=torch.float32, device="cuda") if want_lse else None
    size = kvq.decode_workspace_size_tree(gl.cfg, B, N, Hq)
    if ws is None:
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    held = (bf16_dev(q), bf16_dev(k), bf16_dev(v), dev(np.asarray(parents), torch.int32), gl.seq_lens_dev(lens))
    kvq.decode_attention_tree(gl.cfg, gl.layer.struct(), *held[:4], N, Hq, held[4], B,
                              1 / math.sqrt(128) if scale is None else scale, out, out_bf16, lse, ws, size, gl.status,
                              stream)
    torch.cuda.synchronize()
    return out, lse


def check_tree(out, lse, ref, rlse, slack, half_step=0.0):
    o = out.double().cpu().numpy()
    err, tol = np.abs(o - ref), slack + half_step * (np.abs(ref) + slack) + 2.0 ** -100
    worst, at = float((err / tol).max()), np.unravel_index(np.argmax(err / tol), err.shape)
    assert worst <= 1, (worst, at)


TREES = [
    # fmt, H, g, nodes, kind, lens, G, Gv, R, S, paged, block
    ("int4", 2, 4, 5, "random", [512], 32, 128, 32, 0, False, 16),
    ("int4", 2, 4, 16, "random", [0, 1, 31, 63, 64, 65, 700], 32, 128, 32, 0, False, 16),
    ("int4", 1, 8, 33, "random", [777, 2000, 1], 128, 64, 128, 2, False, 16),      # 264 columns: three chunks
    ("int4", 1, 8, 64, "random", [300], 64, 32, 64, 0, False, 16),                 # 512 columns
    ("int4", 2, 6, 9, "random", [300, 1000, 17, 81], 16, 128, 64, 1, True, 16),
    ("int4", 1, 1, 64, "chain", [1200, 300, 511, 512], 256, 128, 256, 0, False, 16),
    ("int4", 1, 3, 7, "random", [400, 150], 48, 16, 16, 0, False, 16),             # groups that straddle slots
    ("int4", 1, 2, 3, "roots", [400, 333], 80, 128, 0, 3, True, 80),
    ("int8", 2, 6, 3, "random", [300, 17, 80, 81, 2], 16, 128, 64, 1, False, 16),
    ("int8", 3, 2, 20, "star", [250, 96, 97], 16, 32, 64, 1, True, 16),
    ("int8", 1, 8, 16, "random", [900, 767], 256, 16, 32, 1, False, 16),
    ("int2", 3, 1, 32, "random", [1000, 129, 160, 161, 5], 32, 32, 128, 0, False, 16),
    ("int2", 2, 2, 1, "random", [900, 33], 32, 16, 32, 0, True, 32),
    ("int2", 1, 5, 11, "random", [600, 47], 16, 16, 0, 0, False, 16),
    ("fp8_e4m3", 2, 4, 16, "random", [0, 1, 15, 16, 17, 333], 1, 128, 0, 0, False, 16),
    ("fp8_e4m3", 2, 3, 13, "random", [500, 7, 48, 129], 1, 128, 0, 1, True, 16),
    ("fp8_e4m3", 1, 8, 17, "random", [400, 31], 1, 128, 0, 0, True, 48),
    ("fp8_e5m2", 2, 4, 6, "random", [0, 1, 15, 16, 17, 333], 1, 128, 0, 2, False, 16),
    ("fp8_e5m2", 1, 8, 12, "random", [1200, 64], 1, 128, 0, 0, True, 32),
    ("bf16", 2, 4, 5, "random", [0, 1, 15, 16, 17, 333], 0, 0, 0, 0, False, 16),
    ("bf16", 1, 8, 64, "star", [700, 31, 2], 0, 0, 0, 1, False, 16),
    ("bf16", 1, 1, 1, "random", [1500, 160, 127, 128], 0, 0, 0, 3, False, 16),
    # long sequences cut over every SM, merged by the last CTA
    ("int4", 1, 4, 8, "random", [30000], 32, 128, 32, 0, False, 16),
    ("fp8_e4m3", 1, 2, 6, "random", [40000, 12], 1, 128, 0, 1, False, 16),
    ("int2", 1, 8, 10, "random", [25000, 9000], 128, 64, 32, 0, False, 16),
    # more items than SMs
    ("int8", 8, 1, 4, "random", [20 + 13 * i for i in range(24)], 16, 128, 16, 0, False, 16),
]
TREE_IDS = [f"{c[0]}-H{c[1]}g{c[2]}N{c[3]}{c[4]}-G{c[6]}Gv{c[7]}R{c[8]}S{c[9]}{'-paged' if c[10] else ''}" for c in TREES]


@pytest.mark.parametrize("case", TREES, ids=TREE_IDS)
def test_tree_attention(case):
    fmt, H, g, N, kind, lens, G, Gv, R, S_, paged, blk = case
    seed = zlib.crc32(repr(case).encode()) % 10000
    gl, caches = build(fmt, H, lens, G, Gv, R, S_, paged, seed, block_tokens=blk)
    B = len(lens)
    rng = np.random.default_rng(seed)
    q, k, v = draft_inputs(seed, B, H, g, N)
    parents = np.stack([random_tree(rng, N, kind) for _ in range(B)])
    ref, rlse, slack, lslack = S.decode_attention_tree(O.bf16_to_f32(q), caches, O.bf16_to_f32(k), O.bf16_to_f32(v), parents)
    out, lse = tree_call(gl, q, k, v, parents)
    assert gl.status_value() == 0
    check_tree(out, lse, ref, rlse, slack)
    worst = float((np.abs(lse.double().cpu().numpy() - rlse) / lslack).max())
    assert worst <= 1, worst
    out16, lse16 = tree_call(gl, q, k, v, parents, out_bf16=True)
    assert torch.equal(out16, out.to(torch.bfloat16)) and torch.equal(lse16, lse)
    again, _ = tree_call(gl, q, k, v, parents, want_lse=False)
    assert torch.equal(again, out)  # merged in a fixed order


def test_tree_chain_equals_appended_tokens():
    # a chain of drafts = the causal multi-query decode once the drafts are appended (unquantized layer: the
    # appended rows are the drafted ones)
    H, g, N, lens = 2, 2, 4, [333, 5]
    gl, caches = build("bf16", H, lens, 0, 0, 0, 1, False, 7, extra=N)
    q, k, v = draft_inputs(70, 2, H, g, N)
    out, lse = tree_call(gl, q, k, v, np.tile(np.arange(N) - 1, (2, 1)))
    for b in range(2):
        gl.append(b, k[b], v[b], lens[b])
    gl.lens = [T + N for T in lens]
    multi, mlse = gl.decode_multi(q)
    assert gl.status_value() == 0
    # both are held to the oracle elsewhere; their operands differ by f16 / bf16 splits of P: 2^-10 of max|v|
    assert (out - multi).abs().max().item() <= 2 ** -9 * 6 and (lse - mlse).abs().max().item() <= 1e-4


def test_tree_masked_nodes_may_hold_anything():
    # padding nodes with NaN and infinite rows: nobody else sees them
    H, g, N = 2, 4, 6
    for fmt in ("int4", "fp8_e4m3", "bf16"):
        fp8 = fmt == "fp8_e4m3"
        gl, caches = build(fmt, H, [100, 3], 1 if fp8 else 32, 128, 0 if fp8 else 32, 0, False, 11)
        q, k, v = draft_inputs(5, 2, H, g, N)
        parents = np.array([[-1, 0, 1, -1, -1, 0], [-1, 0, 0, 2, -1, 3]])
        ref, rlse, slack, lslack = S.decode_attention_tree(O.bf16_to_f32(q), caches, O.bf16_to_f32(k), O.bf16_to_f32(v), parents)
        k2, v2 = k.copy(), v.copy()
        for b, n in ((0, 3), (0, 4), (1, 4)):
            k2[b, :, n] = 0x7FC0
            v2[b, :, n, ::2] = 0x7F80
            v2[b, :, n, 1::2] = 0xFFC0
        out, lse = tree_call(gl, q, k2, v2, parents)
        assert gl.status_value() == kvq.DEV_RANGE
        keep = np.ones((2, N), bool)
        for b, n in ((0, 3), (0, 4), (1, 4)):
            keep[b, n] = False
        o = out.double().cpu().numpy()
        assert np.all(np.abs(o - ref)[keep] <= slack[keep])
        assert np.isnan(o[~keep]).all()
        # a Value alone beyond f16: the nodes that see it are not numbers, the others are untouched
        gl.status.zero_()
        v3 = v.copy()
        v3[0, :, 1, 7] = I.f32_to_bf16_bits(np.array([1e30], F32))[0]
        out, _ = tree_call(gl, q, k, v3, parents)
        o = out.double().cpu().numpy()
        assert gl.status_value() == kvq.DEV_RANGE
        assert np.isnan(o[0, [1, 2]]).all()
        rest = [0, 3, 4, 5]
        assert np.all(np.abs(o - ref)[0, rest] <= slack[0, rest]) and np.all(np.abs(o - ref)[1] <= slack[1])


def test_tree_reports_bad_inputs_and_carries_on():
    H, g, N = 2, 2, 5
    gl, caches = build("int4", H, [200, 130, 90], 16, 128, 16, 0, True, 3)
    q, k, v = draft_inputs(9, 3, H, g, N)
    parents = np.array([[-1, 0, 5, -7, 3], [-1, 0, 1, 2, 3], [0, 0, 0, 0, 0]])
    fixed = np.array([[-1, 0, -1, -1, 3], [-1, 0, 1, 2, 3], [-1, 0, 0, 0, 0]])
    args = (O.bf16_to_f32(q), caches, O.bf16_to_f32(k), O.bf16_to_f32(v), fixed)
    ref, rlse, slack, lslack = S.decode_attention_tree(*args)
    out, lse = tree_call(gl, q, k, v, parents)
    assert gl.status_value() == kvq.DEV_BAD_TREE
    check_tree(out, lse, ref, rlse, slack)
    # a block outside the pool: its tokens are left out
    gl.status.zero_()
    table = gl.layer.block_table.clone()
    gl.layer.block_table[0, 2], gl.layer.block_table[1, 0] = 10 ** 6, -3
    out, lse = tree_call(gl, q, k, v, fixed)
    assert gl.status_value() == kvq.DEV_BAD_BLOCK
    gl.layer.block_table.copy_(table)
    for b, cut in ((0, 2), (1, 0)):
        for h in range(H):
            kk, vv = O.attention_keys(caches[b][h])
            left = np.r_[0:16 * cut, 16 * cut + 16:len(kk)]
            for n in range(N):
                seen = S.ancestors(fixed[b])[n]
                ka = np.concatenate([kk[left], O.bf16_to_f32(k[b, h])[seen]])
                va = np.concatenate([vv[left], O.bf16_to_f32(v[b, h])[seen]])
                for j in range(g):
                    o, _ = O.attend_head(O.bf16_to_f32(q[b, n, h * g + j]), ka, va, 1 / math.sqrt(128))
                    # (the slack of the whole sequence, widened by the probability that the cut block held)
                    assert np.abs(out[b, n, h * g + j].double().cpu().numpy() - o).max() <= 4 * slack[b, n].max()
    # a length beyond the store is cut to it, a negative one counts as empty
    gl.status.zero_()
    cap = gl.mbps * 16 + 16 + 15
    out, _ = tree_call(gl, q, k, v, fixed, lens=[200, 130, -5])
    empty = [[O.empty_head_cache(gl.spec) for _ in range(H)] for _ in range(3)]
    ref2, rl2, slack2, _ = S.decode_attention_tree(args[0], empty, *args[2:])
    assert np.all(np.abs(out.double().cpu().numpy() - ref2)[2] <= slack2[2]) and gl.status_value() == 0
    tree_call(gl, q, k, v, fixed, lens=[cap + 1, 130, 90])
    assert gl.status_value() & kvq.DEV_CAPACITY


def test_tree_key_scales_beyond_f16_are_reported():
    gl, caches = build("int4", 1, [200], 32, 128, 32, 0, False, 3)
    q, k, v = draft_inputs(9, 1, 1, 2, 3)
    parents = np.array([[-1, 0, 1]])
    store = gl.layer.buf["qstore"]
    store[:512].view(torch.float32)[5] = 3e4  # a Key scale: 15 steps of it leave f16
    tree_call(gl, q, k, v, parents)
    assert gl.status_value() == kvq.DEV_RANGE
    gl.status.zero_()
    q2 = q.copy()
    q2[0, 1, 0, 3] = I.f32_to_bf16_bits(np.array([7e4], F32))[0]
    gl, caches = build("int4", 1, [200], 32, 128, 32, 0, False, 3)
    tree_call(gl, q2, k, v, parents)
    assert gl.status_value() == kvq.DEV_RANGE


def test_tree_extreme_scores_and_scales():
    # scores that rise along the sequence (the maximum moves again and again), very negative ones, scale 0
    H, g, N, T = 1, 4, 8, 1500
    rng = np.random.default_rng(2)
    for factor in (40.0, -40.0):
        gl = TL.GpuLayer("bf16", H, [T], 0, 0, 0, 0, seed=1)
        base = I.bf16_bits_to_f32(I.random_bf16(3, (128,)))
        ramp = np.linspace(0, 1, T)[:, None]
        k = I.f32_to_bf16_bits((base * ramp * factor / 11 + 0.1 * rng.standard_normal((T, 128))).astype(F32))
        v = I.random_bf16(4, (T, 128))
        gl.append(0, k[None], v[None], 0)
        caches = [[O.build_head_cache(O.bf16_to_f32(k), O.bf16_to_f32(v), gl.spec)]]
        q, kd, vd = draft_inputs(6, 1, H, g, N)
        q = I.f32_to_bf16_bits((base + 0.2 * I.bf16_bits_to_f32(q)).astype(F32))
        parents = np.array([random_tree(rng, N, "random")])
        args = (O.bf16_to_f32(q), caches, O.bf16_to_f32(kd), O.bf16_to_f32(vd), parents)
        for scale in (1 / math.sqrt(128), 2.0, 0.0, -0.05):
            ref, rlse, slack, lslack = S.decode_attention_tree(*args, scale=scale)
            out, lse = tree_call(gl, q, kd, vd, parents, scale=scale)
            check_tree(out, lse, ref, rlse, slack)
            worst = float((np.abs(lse.double().cpu().numpy() - rlse) / lslack).max())
            assert worst <= 1, worst


def test_tree_workspace_is_left_ready_and_streams_and_graphs_work():
    H, g, N = 2, 4, 7
    gl, caches = build("int4", H, [9000, 40, 3000], 32, 128, 32, 0, False, 21)
    q, k, v = draft_inputs(2, 3, H, g, N)
    parents = np.stack([random_tree(np.random.default_rng(i), N, "random") for i in range(3)])
    want, _ = tree_call(gl, q, k, v, parents)
    size = kvq.decode_workspace_size_tree(gl.cfg, 3, N, H * g)
    # one workspace, used again and again, on a stream of its own, then from a captured graph
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    held = (bf16_dev(q), bf16_dev(k), bf16_dev(v), dev(parents, torch.int32), gl.seq_lens_dev())
    outs = [torch.empty_like(want) for _ in range(3)]
    torch.cuda.synchronize()
    call = lambda out, stream: kvq.decode_attention_tree(  # noqa: E731
        gl.cfg, gl.layer.struct(), *held[:4], N, H * g, held[4], 3, 1 / math.sqrt(128), out, False, None, ws, size,
        gl.status, stream)
    for o in outs:
        call(o, side)
    side.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph, o = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        call(o, torch.cuda.current_stream())
        call(outs[0], torch.cuda.current_stream())
    for _ in range(2):
        o.zero_(), outs[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(outs[0], want)
    assert gl.status_value() == 0
    with pytest.raises(kvq.KvqError) as e:
        kvq.decode_attention_tree(gl.cfg, gl.layer.struct(), *held[:4], N, H * g, held[4], 3, 0.1, o, False, None, ws,
                                  size - 1, gl.status)
    assert e.value.status == -4


# --------------------------------------------------------------------------- #
# verification
# --------------------------------------------------------------------------- #


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(F32)


def verify_call(target, draft, tokens, parents, u, pad=0):
    B, N, V = target.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = [None if a is None else dev(np.concatenate([a, np.full((B, N, pad), np.nan, F32)], -1))
            for a in (target, draft)]
    path = torch.full((B, N), -9, dtype=torch.int32, device="cuda")
    acc, nxt = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    kvq.verify_tree(wide[0], V + pad, wide[1], V + pad, V, dev(tokens, torch.int32), dev(parents, torch.int32),
                    dev(u.astype(F32)), N, B, path, acc, nxt, st)
    torch.cuda.synchronize()
    return path.cpu().numpy(), acc.cpu().numpy(), nxt.cpu().numpy(), int(st.item())


def check_verify(target, draft, tokens, parents, u, got):
    path, acc, nxt, _ = got
    for b in range(target.shape[0]):
        rp, rn = S.verify_tree(target[b], None if draft is None else draft[b], tokens[b], parents[b], u[b].astype(F32))
        assert list(path[b]) == rp + [-1] * (path.shape[1] - len(rp)) and acc[b] == len(rp) and nxt[b] == rn, (b, rp, rn)


VERIFY = [  # batch, nodes, vocab, drafted, kind, pad
    (1, 1, 1, True, "chain", 0), (3, 1, 50, True, "chain", 0), (4, 6, 2, True, "chain", 1), (5, 9, 33, False, "random", 0),
    (64, 8, 1000, True, "random", 3), (64, 8, 1000, False, "random", 0), (2, 64, 4099, True, "random", 5),
    (1, 6, 32000, True, "chain", 0), (7, 5, 128256, True, "star", 0), (300, 4, 517, True, "star", 0),
]


@pytest.mark.parametrize("case", VERIFY, ids=[f"B{c[0]}N{c[1]}V{c[2]}{c[4]}{'' if c[3] else '-chosen'}" for c in VERIFY])
def test_verify_tree(case):
    B, N, V, drafted, kind, pad = case
    rng = np.random.default_rng(zlib.crc32(repr(case).encode()))
    logits = 2.5 * rng.standard_normal((B, N, V))
    target, draft = softmax(logits), softmax(logits + 1.5 * rng.standard_normal((B, N, V)))
    parents = np.stack([random_tree(rng, N, kind) for _ in range(B)])
    tokens = np.zeros((B, N), np.int64)
    for b in range(B):
        for n in range(1, N):
            pr = draft[b, max(parents[b, n], 0)].astype(np.float64)
            tokens[b, n] = rng.choice(V, p=pr / pr.sum())
    u = rng.random((B, N)).astype(F32)
    u[0, 0] = 0.0
    u[B - 1, 0] = 1.0 - 2.0 ** -24
    d = draft if drafted else None
    got = verify_call(target, d, tokens, parents, u, pad)
    assert got[3] == 0
    check_verify(target, d, tokens, parents, u, got)
    assert all(np.array_equal(a, b) for a, b in zip(got, verify_call(target, d, tokens, parents, u, pad)))


def test_verify_tree_edges():
    rng = np.random.default_rng(8)
    B, N, V = 6, 4, 3001
    target, draft = (softmax(2 * rng.standard_normal((B, N, V))) for _ in range(2))
    parents = np.tile([-1, 0, 0, 1], (B, 1))
    tokens = rng.integers(0, V, (B, N))
    u = rng.random((B, N)).astype(F32)
    draft[1] = target[1]                       # the same distributions: the first child is accepted
    target[2, 0], draft[2, 0] = 0, 0           # one token each: nothing left after a rejection
    target[2, 0, 7], draft[2, 0, 9] = 1, 1
    tokens[2] = [0, 9, 9, 9]
    target[3] = 0                              # no distribution at all
    target[4, :, 5] = np.nan
    tokens[5] = [0, V, -1, 0]                  # tokens that do not exist
    got = verify_call(target, draft, tokens, parents, u)
    assert got[3] == kvq.DEV_BAD_TREE | kvq.DEV_BAD_PROBS
    keep = [0, 1, 2, 3, 5]
    check_verify(target[keep], draft[keep], tokens[keep], parents[keep], u[keep], [a[keep] for a in got[:3]] + [0])
    assert got[2][2] == 7 and got[2][3] == -1 and got[2][4] == -1 and got[1][1] >= 2
    bad = np.tile([-1, 3, -4, 0], (B, 1))      # parents out of range count as none
    got = verify_call(target[:2], draft[:2], tokens[:2], bad[:2], u[:2])
    assert got[3] == kvq.DEV_BAD_TREE
    check_verify(target[:2], draft[:2], tokens[:2], np.tile([-1, -1, -1, 0], (2, 1)), u[:2], got)
    # numbers outside [0, 1): 1 and NaN draw the last token with weight and accept nothing
    for x in (1.0, np.nan):
        ux = np.full((2, N), x, F32)
        got = verify_call(target[:2], draft[:2], tokens[:2], parents[:2], ux)
        assert list(got[1]) == [1 if x != x else got[1][0], 1 if x != x else got[1][1]]
        check_verify(target[:2], draft[:2], tokens[:2], parents[:2], ux, got)


# --------------------------------------------------------------------------- #
# append of the accepted path
# --------------------------------------------------------------------------- #

APPEND = [
    ("int4", 2, [0, 1, 40, 63, 64, 100], 32, 128, 32, 0, False, 9),
    ("int4", 2, [70, 15, 31], 16, 64, 0, 2, True, 40),     # several groups spill at once
    ("int8", 1, [200, 255, 240], 128, 32, 128, 1, False, 64),
    ("int2", 3, [90, 5, 64], 32, 16, 16, 0, False, 33),
    ("fp8_e4m3", 2, [0, 15, 16, 30, 77], 1, 128, 0, 0, False, 20),
    ("fp8_e5m2", 1, [3, 47], 1, 128, 0, 5, True, 17),
    ("bf16", 2, [0, 1, 130], 0, 0, 0, 3, False, 8),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"{c[0]}-G{c[3]}R{c[5]}S{c[6]}{'-paged' if c[7] else ''}" for c in APPEND])
def test_append_accepted(case):
    fmt, H, lens, G, Gv, R, S_, paged, N = case
    seed = zlib.crc32(repr(case).encode()) % 10000
    gl, caches = build(fmt, H, lens, G, Gv, R, S_, paged, seed, extra=N)
    B = len(lens)
    rng = np.random.default_rng(seed)
    _, k, v = draft_inputs(seed, B, H, 1, N)
    counts = np.array([[N, 0, 1, N // 2, N - 1, 3][b % 6] for b in range(B)])
    path = np.full((B, N), -1)
    for b in range(B):
        path[b, :counts[b]] = np.sort(rng.choice(N, counts[b], replace=False))
    path[0, :counts[0]] = rng.permutation(N)[:counts[0]]  # any order, and the same row twice
    if N > 2:
        path[0, 1] = path[0, 0]
    kvq.append_accepted(gl.cfg, gl.layer.struct(), bf16_dev(k), bf16_dev(v), N, dev(path, torch.int32),
                        dev(counts, torch.int32), gl.seq_lens_dev(), B, gl.status)
    torch.cuda.synchronize()
    assert gl.status_value() == 0
    for b in range(B):
        for h in range(H):
            for j in range(counts[b]):
                O.append_token(caches[b][h], O.bf16_to_f32(k[b, h, path[b, j]]), O.bf16_to_f32(v[b, h, path[b, j]]))
            TL.compare_logical(gl.logical(b, h, lens[b] + int(counts[b])), caches[b][h])


def test_append_accepted_leaves_bad_sequences_alone():
    for fmt, G, R in (("int4", 16, 16), ("fp8_e4m3", 1, 0), ("bf16", 0, 0)):
        H, lens, N = 2, [40, 33, 20, 8], 6
        gl, caches = build(fmt, H, lens, G, 128, R, 0, False, 5, extra=N)
        _, k, v = draft_inputs(1, 4, H, 1, N)
        path = np.array([[0, 1, 6, -1, -1, -1], [0, -2, 2, -1, -1, -1], [0, 1, 2, 3, 4, 5], [5, 4, -1, -1, -1, -1]])
        counts = np.array([3, 2, 7, 2])
        kvq.append_accepted(gl.cfg, gl.layer.struct(), bf16_dev(k), bf16_dev(v), N, dev(path, torch.int32),
                            dev(counts, torch.int32), gl.seq_lens_dev(), 4, gl.status)
        torch.cuda.synchronize()
        assert gl.status_value() == kvq.DEV_BAD_TREE
        for b in range(4):
            for h in range(H):
                if b == 3:
                    for j in range(2):
                        O.append_token(caches[b][h], O.bf16_to_f32(k[b, h, path[b, j]]), O.bf16_to_f32(v[b, h, path[b, j]]))
                TL.compare_logical(gl.logical(b, h, lens[b] + (2 if b == 3 else 0)), caches[b][h])
        # no room: nothing is written, the others are
        gl.status.zero_()
        many = np.array([N, N, N, N])
        long = gl.seq_lens_dev([40, 10 ** 6, 20, 8])
        before = {n: t.clone() for n, t in gl.layer.buf.items() if t is not None}
        kvq.append_accepted(gl.cfg, gl.layer.seq_struct(1), bf16_dev(k[1:2]), bf16_dev(v[1:2]), N,
                            dev(np.arange(N)[None], torch.int32), dev(many[:1], torch.int32), long[1:2], 1, gl.status)
        torch.cuda.synchronize()
        assert gl.status_value() == kvq.DEV_CAPACITY
        assert all(torch.equal(t, gl.layer.buf[n]) for n, t in before.items())


# --------------------------------------------------------------------------- #
# a run of the four together, as a decoding loop makes it
# --------------------------------------------------------------------------- #


@pytest.mark.parametrize("fmt", ["int4", "int2", "fp8_e4m3", "bf16"])
def test_decoding_steps(fmt):
    """Three speculative steps of a one-layer toy model on the device, no host work in between but reading the
    results for the oracle: projection rows -> norm and rotation -> tree attention -> verification -> append."""
    fp8 = fmt.startswith("fp8")
    B, H, g, N, V, lens, base, eps = 3, 2, 3, 7, 211, [70, 33, 1], 10000.0, 1e-6
    G, R = (1, 0) if fp8 else (16, 16)
    gl, caches = build(fmt, H, lens, G, 128, R, 1, False, 31, extra=3 * N)
    rng = np.random.default_rng(17)
    w = [bf16_dev(I.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(128)).astype(F32))) for _ in range(2)]
    seq = gl.seq_lens_dev()
    size = kvq.decode_workspace_size_tree(gl.cfg, B, N, H * g)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, out = torch.empty(B, N, H * g, 128, **bf), torch.empty(B, N, H * g, 128, dtype=torch.float32, device="cuda")
    k, v = torch.empty(B, H, N, 128, **bf), torch.empty(B, H, N, 128, **bf)
    path, acc, nxt = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B, N), (B,), (B,)))
    for step in range(3):
        parents = np.stack([random_tree(rng, N, "random") for _ in range(B)])
        parents[:, 1:][parents[:, 1:] < 0] = 0
        depth = np.zeros((B, N), np.int32)
        for n in range(1, N):
            depth[:, n] = depth[np.arange(B), parents[:, n]] + 1
        rows = bf16_dev(I.random_bf16(100 + step, (B * N, (H * g + 2 * H) * 128)))
        pd = dev(parents, torch.int32)
        positions = (seq[:, None] + dev(depth)).int().contiguous()
        kvq.qk_norm_rope(rows, rows.shape[1], B, N, H * g, H, *w, eps, positions, base, True, q, k, v)
        kvq.decode_attention_tree(gl.cfg, gl.layer.struct(), q, k, v, pd, N, H * g, seq, B, 1 / math.sqrt(128), out, False,
                                  None, ws, size, gl.status)
        # toy logits from the attention output: one set of random vectors as the head
        head = dev(rng.standard_normal((H * g * 128, V)).astype(F32) / 8)
        target = (out.reshape(B, N, -1) @ head).softmax(-1).contiguous()
        draft = (target.log() + dev(rng.standard_normal((B, N, V)).astype(F32))).softmax(-1).contiguous()
        tokens = dev(rng.integers(0, V, (B, N)), torch.int32)
        best = draft.argmax(-1).int()  # likely children, so that paths get long
        tokens[:, 1:] = best.gather(1, pd[:, 1:].long())
        u = dev(rng.random((B, N)).astype(F32))
        kvq.verify_tree(target, V, draft, V, V, tokens, pd, u, N, B, path, acc, nxt, gl.status)
        kvq.append_accepted(gl.cfg, gl.layer.struct(), k, v, N, path, acc, seq, B, gl.status)
        old = seq.cpu().numpy()
        seq += acc
        torch.cuda.synchronize()
        assert gl.status_value() == 0
        qb, kb, vb = bits_of(q), bits_of(k), bits_of(v)
        ref, rlse, slack, lslack = S.decode_attention_tree(O.bf16_to_f32(qb), caches, O.bf16_to_f32(kb), O.bf16_to_f32(vb), parents)
        check_tree(out, None, ref, rlse, slack)
        pa, ac, nx = path.cpu().numpy(), acc.cpu().numpy(), nxt.cpu().numpy()
        check_verify(target.cpu().numpy(), draft.cpu().numpy(), tokens.cpu().numpy(), parents, u.cpu().numpy(),
                     (pa, ac, nx, 0))
        for b in range(B):
            for h in range(H):
                for n in pa[b, :ac[b]]:
                    O.append_token(caches[b][h], O.bf16_to_f32(kb[b, h, n]), O.bf16_to_f32(vb[b, h, n]))
                TL.compare_logical(gl.logical(b, h, int(old[b] + ac[b])), caches[b][h])
    assert (seq.cpu().numpy() > np.array(lens) + 2).all()


def test_tree_reads_blocks_beyond_4_gib():
    # a pool of 420000 blocks (4.4 GB), the sequences' blocks scattered over it
    H, g, N = 2, 2, 6
    gl = TL.GpuLayer("int8", H, [333, 90], 16, 128, 16, 0, paged=True, seed=5, spare_blocks=420000)
    assert gl.layer.sizes["block_pool"] > 1 << 32
    table = gl.layer.block_table
    used = table >= 0
    table[used] = (gl.cfg.num_blocks - 1 - 7 * torch.arange(int(used.sum()), device="cuda")).int()
    rng = np.random.default_rng(0)
    kv = [[(I.random_bf16(10 * b + h, (T, 128)), I.random_bf16(50 + 10 * b + h, (T, 128))) for h in range(H)]
          for b, T in enumerate(gl.lens)]
    for b in range(2):
        gl.append(b, np.stack([kv[b][h][0] for h in range(H)]), np.stack([kv[b][h][1] for h in range(H)]), 0)
    caches = [[O.build_head_cache(O.bf16_to_f32(k), O.bf16_to_f32(v), gl.spec) for k, v in row] for row in kv]
    q, k, v = draft_inputs(8, 2, H, g, N)
    parents = np.stack([random_tree(rng, N, "random") for _ in range(2)])
    ref, rlse, slack, lslack = S.decode_attention_tree(O.bf16_to_f32(q), caches, O.bf16_to_f32(k), O.bf16_to_f32(v), parents)
    out, lse = tree_call(gl, q, k, v, parents)
    assert gl.status_value() == 0
    check_tree(out, lse, ref, rlse, slack)


@pytest.mark.parametrize("lens", [[700] * 5, [5] * 40 + [1500], [130, 2000, 1, 0, 640, 90]])
@pytest.mark.parametrize("fmt", ["int4", "fp8_e5m2"])
def test_tree_work_split(fmt, lens):
    # equal lengths (whole items), many short ones (a CTA each), ragged ones (cut and merged), with sequences of very
    # different size side by side; two chunks of columns
    H, g, N = 2, 8, 17
    fp8 = fmt.startswith("fp8")
    gl, caches = build(fmt, H, lens, 1 if fp8 else 32, 128, 0 if fp8 else 64, 1, False, len(lens))
    rng = np.random.default_rng(4)
    B = len(lens)
    q, k, v = draft_inputs(40, B, H, g, N)
    parents = np.stack([random_tree(rng, N, "random") for _ in range(B)])
    ref, rlse, slack, lslack = S.decode_attention_tree(O.bf16_to_f32(q), caches, O.bf16_to_f32(k), O.bf16_to_f32(v), parents)
    out, lse = tree_call(gl, q, k, v, parents)
    assert gl.status_value() == 0
    check_tree(out, lse, ref, rlse, slack)
    worst = float((np.abs(lse.double().cpu().numpy() - rlse) / lslack).max())
    assert worst <= 1, worst


def test_calls_on_another_stream_and_in_a_graph():
    # norm and rotation, verification and append on a side stream and captured: the results of the plain calls
    B, n, hq, h, V = 3, 5, 8, 2, 3001
    rng = np.random.default_rng(12)
    rows = bf16_dev(I.random_bf16(1, (B * n, (hq + 2 * h) * 128)))
    w = [bf16_dev(I.random_bf16(2 + i, (128,))) for i in range(2)]
    pos = dev(rng.integers(0, 9000, (B, n)), torch.int32)
    target, draft = (dev(softmax(2 * rng.standard_normal((B, n, V)))) for _ in range(2))
    tokens, parents = dev(rng.integers(0, V, (B, n)), torch.int32), dev(np.tile(np.arange(n) - 1, (B, 1)), torch.int32)
    u = dev(rng.random((B, n)).astype(F32))
    gl, _ = build("int4", h, [100, 40, 63], 32, 128, 32, 0, False, 8, extra=n)
    seq = gl.seq_lens_dev()
    start = {k: t.clone() for k, t in gl.layer.buf.items() if t is not None}

    def buffers():
        bf = dict(dtype=torch.bfloat16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        return (torch.zeros(B, n, hq, 128, **bf), torch.zeros(B, h, n, 128, **bf), torch.zeros(B, h, n, 128, **bf),
                torch.zeros(B, n, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32))

    def step(o, stream=None):
        kvq.qk_norm_rope(rows, rows.shape[1], B, n, hq, h, *w, 1e-6, pos, 1e4, True, *o[:3], stream=stream)
        kvq.verify_tree(target, V, draft, V, V, tokens, parents, u, n, B, *o[3:], gl.status, stream=stream)
        kvq.append_accepted(gl.cfg, gl.layer.struct(), o[1], o[2], n, o[3], o[4], seq, B, gl.status, stream=stream)

    def restore():
        for k, t in start.items():
            gl.layer.buf[k].copy_(t)
        torch.cuda.synchronize()

    want = buffers()
    step(want)
    torch.cuda.synchronize()
    held = {k: gl.layer.buf[k].clone() for k in start}
    restore()
    side, o = torch.cuda.Stream(), buffers()
    torch.cuda.synchronize()
    step(o, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, want)) and all(torch.equal(gl.layer.buf[k], t) for k, t in held.items())
    restore()
    graph, o = torch.cuda.CUDAGraph(), buffers()
    with torch.cuda.graph(graph):
        step(o)
    for _ in range(2):
        restore()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want))
        assert all(torch.equal(gl.layer.buf[k], t) for k, t in held.items())
    assert gl.status_value() == 0


def test_two_tree_calls_at_once():
    # two streams, a workspace each, cut sequences of different size: each gets what it gets alone
    H, g, N = 2, 4, 7
    gl, caches = build("int4", H, [20000, 40, 6000], 32, 128, 32, 0, False, 21)
    runs = []
    for i, lens in enumerate(([20000, 40, 6000], [9000, 33, 1])):
        q, k, v = draft_inputs(60 + i, 3, H, g, N)
        parents = np.stack([random_tree(np.random.default_rng(10 * i + j), N, "random") for j in range(3)])
        want, _ = tree_call(gl, q, k, v, parents, lens=lens)
        size = kvq.decode_workspace_size_tree(gl.cfg, 3, N, H * g)
        runs.append((want, [torch.zeros_like(want) for _ in range(8)], torch.zeros(size, dtype=torch.uint8, device="cuda"),
                     size, (bf16_dev(q), bf16_dev(k), bf16_dev(v), dev(parents, torch.int32), gl.seq_lens_dev(lens)),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for j in range(8):
        for _, outs, ws, size, held, stream in runs:
            kvq.decode_attention_tree(gl.cfg, gl.layer.struct(), *held[:4], N, H * g, held[4], 3, 1 / math.sqrt(128),
                                      outs[j], False, None, ws, size, gl.status, stream)
    torch.cuda.synchronize()
    assert gl.status_value() == 0
    assert all(torch.equal(o, want) for want, outs, *_ in runs for o in outs)


def test_tree_query_that_is_not_a_number():
    # a row of NaN gives NaN whether its sequence is cut over CTAs or not; the other rows keep their results
    H, g, N = 1, 2, 4
    gl, caches = build("int4", H, [6000, 70], 32, 128, 32, 0, False, 13)
    q, k, v = draft_inputs(3, 2, H, g, N)
    parents = np.tile([-1, 0, 1, 0], (2, 1))
    want, wlse = tree_call(gl, q, k, v, parents)
    q2 = q.copy()
    q2[:, 2, 1] = 0x7FC0
    out, lse = tree_call(gl, q2, k, v, parents)
    assert gl.status_value() == kvq.DEV_RANGE
    bad = torch.zeros(2, N, H * g, dtype=torch.bool, device="cuda")
    bad[:, 2, 1] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], wlse[~bad])
