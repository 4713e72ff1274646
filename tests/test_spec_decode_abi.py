"""Speculative decoding calls on the CPU: the oracle's own pins, and every refusal that the host makes
before anything is enqueued (the pointers below are fake, aligned and never dereferenced)."""
import numpy as np
import pytest

from oracle import spec_oracle as S


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_decode_gb300 as pkg
    pkg.build()
    from quantized_kv_cache_decode_gb300 import kvq as mod
    return mod


def status_of(kvq, call):
    with pytest.raises(kvq.KvqError) as e:
        call()
    return e.value.status


ROPE = dict(qkv=4096, row_stride=12 * 128, batch=2, n_tokens=3, num_q_heads=8, num_kv_heads=2, q_weight=8192,
            k_weight=None, eps=1e-6, positions=4, rope_base=1e4, rotate_keys=1, q_out=16, k_out=32, v_out=48)


@pytest.mark.parametrize("bad,status", [
    (dict(row_stride=12 * 128 - 8), -1), (dict(row_stride=12 * 128 + 4), -1), (dict(batch=-1), -1),
    (dict(n_tokens=-1), -1), (dict(num_q_heads=0), -1), (dict(num_kv_heads=0), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(rope_base=1.0), -1),
    (dict(rope_base=float("nan")), -1), (dict(rotate_keys=2), -1), (dict(qkv=0), -1), (dict(qkv=4100), -1),
    (dict(q_out=0), -1), (dict(k_out=8), -1), (dict(v_out=0), -1), (dict(positions=None), -1),
    (dict(q_weight=8194), -1), (dict(k_weight=8200), -1), (dict(head_dim=64), -2),
    (dict(batch=1 << 16, n_tokens=1 << 15), -2)])
def test_qk_norm_rope_refusals(kvq, bad, status):
    assert status_of(kvq, lambda: kvq.qk_norm_rope(**{**ROPE, **bad}, stream=0)) == status


def test_qk_norm_rope_empty_batches_do_nothing(kvq):
    kvq.qk_norm_rope(**{**ROPE, "batch": 0, "qkv": 0}, stream=0)
    kvq.qk_norm_rope(**{**ROPE, "n_tokens": 0, "qkv": 0}, stream=0)


VERIFY = dict(target_probs=16, target_stride=100, draft_probs=16, draft_stride=100, vocab=100, tokens=16, parents=16,
              uniforms=16, n_nodes=4, batch=2, path=16, n_accepted=16, next_token=16)


@pytest.mark.parametrize("bad", [dict(vocab=0), dict(n_nodes=0), dict(n_nodes=65), dict(batch=-1), dict(batch=2049),
                                 dict(target_stride=99), dict(draft_stride=99), dict(target_probs=None),
                                 dict(tokens=None), dict(parents=None), dict(uniforms=None), dict(path=None),
                                 dict(n_accepted=None), dict(next_token=None)])
def test_verify_tree_refusals(kvq, bad):
    assert status_of(kvq, lambda: kvq.verify_tree(**{**VERIFY, **bad}, stream=0)) == -1


def test_verify_tree_refuses_rows_beyond_its_counters(kvq):
    wide = dict(vocab=(1 << 30) + 1, target_stride=1 << 31, draft_stride=1 << 31)
    assert status_of(kvq, lambda: kvq.verify_tree(**{**VERIFY, **wide}, stream=0)) == -2


def test_verify_tree_without_sequences_does_nothing(kvq):
    kvq.verify_tree(**{**VERIFY, "batch": 0}, stream=0)


def layer(kvq, fmt="int4", **kw):
    fp8 = fmt.startswith("fp8")
    cfg = kvq.make_config(fmt, 2, 1 if fp8 else 32, 128, 0 if fp8 else 32, 0, capacity_tokens=64, **kw)
    cache = kvq.LayerCache()
    cache.qstore, cache.resid_k, cache.resid_v = 1 << 20, 2 << 20, 3 << 20
    cache.k_tensor_scale = cache.v_tensor_scale = 4096
    return cfg, cache


@pytest.mark.parametrize("bad,status", [
    (dict(n_nodes=0), -1), (dict(n_nodes=65), -1), (dict(batch=-1), -1), (dict(batch=2049), -1),
    (dict(num_q_heads=3), -1), (dict(num_q_heads=18), -1), (dict(out_bf16=2), -1), (dict(q=8), -1), (dict(q=0), -1),
    (dict(k_draft=0), -1), (dict(v_draft=24), -1), (dict(parents=0), -1), (dict(seq_lens=0), -1), (dict(out=0), -1), (dict(out=4104), -1),
    (dict(softmax_scale=float("nan")), -1), (dict(workspace=0), -1), (dict(workspace=8), -1)])
def test_decode_attention_tree_refusals(kvq, bad, status):
    cfg, cache = layer(kvq)
    a = dict(q=4096, k_draft=4096, v_draft=4096, parents=16, n_nodes=5, num_q_heads=8, seq_lens=16, batch=2,
             softmax_scale=0.1, out=4096, out_bf16=0, lse=0, workspace=4096, workspace_bytes=1 << 40)
    assert status_of(kvq, lambda: kvq.decode_attention_tree(cfg, cache, **{**a, **bad}, stream=0)) == status


def test_decode_attention_tree_refuses_layers_it_does_not_read(kvq):
    for kw in (dict(rope_base=1e4), dict(k_outliers=1), dict(v_outliers=2)):
        cfg, cache = layer(kvq, **kw)
        assert status_of(kvq, lambda: kvq.decode_attention_tree(cfg, cache, 4096, 4096, 4096, 16, 5, 8, 16, 2, 0.1, 4096,
                                                                0, 0, 4096, 1 << 40, stream=0)) == -2
        assert status_of(kvq, lambda: kvq.decode_workspace_size_tree(cfg, 2, 5, 8)) == -2
    cfg, cache = layer(kvq)
    cache.resid_v = None
    assert status_of(kvq, lambda: kvq.decode_attention_tree(cfg, cache, 4096, 4096, 4096, 16, 5, 8, 16, 2, 0.1, 4096, 0,
                                                            0, 4096, 1 << 40, stream=0)) == -1


@pytest.mark.parametrize("bad", [dict(n_nodes=0), dict(n_nodes=65), dict(batch=-1), dict(k_draft=0), dict(k_draft=8),
                                 dict(v_draft=4), dict(path=0), dict(n_accepted=0), dict(seq_lens=0)])
def test_append_accepted_refusals(kvq, bad):
    cfg, cache = layer(kvq)
    a = dict(k_draft=4096, v_draft=4096, n_nodes=5, path=16, n_accepted=16, seq_lens=16, batch=2)
    assert status_of(kvq, lambda: kvq.append_accepted(cfg, cache, **{**a, **bad}, stream=0)) == -1


# --------------------------------------------------------------------------- #
# the oracle's pins
# --------------------------------------------------------------------------- #


def test_oracle_ancestors():
    seen = S.ancestors([-1, 0, 0, 1, -1, 3])
    assert [list(np.nonzero(r)[0]) for r in seen] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [0, 1, 3, 5]]


def test_oracle_rotation_is_the_cache_oracles():
    from oracle import kvq_oracle as O
    x = np.random.default_rng(0).standard_normal((5, 128))
    pos = np.array([0, 1, 17, 4095, 100000])
    assert np.allclose(S.rotate_exact(x, pos, 10000.0), O.rope_rotate(x, pos, 10000.0), atol=1e-9)


@pytest.mark.parametrize("drawn", [True, False])
def test_oracle_verification_keeps_the_target_distribution(drawn):
    # the first emitted token (the first accepted child's, or the drawn one) must follow the target
    # whatever the drafter: 20000 trials of a root with three children, V = 5.  Each frequency's
    # standard deviation is at most sqrt(1/4 / 20000) = 0.0036; five of them are 0.018
    rng = np.random.default_rng(5)
    p, q = np.array([0.4, 0.25, 0.2, 0.1, 0.05]), np.array([0.1, 0.5, 0.1, 0.1, 0.2])
    target, draft = np.tile(p, (4, 1)), np.tile(q, (4, 1))
    n, count = 20000, np.zeros(5)
    for _ in range(n):
        tokens = np.array([0, *(rng.choice(5, 3, p=q) if drawn else rng.permutation(5)[:3])])
        path, nxt = S.verify_tree(target, draft if drawn else None, tokens, [-1, 0, 0, 0], rng.random(4))
        count[tokens[path[1]] if len(path) > 1 else nxt] += 1
    assert np.abs(count / n - p).max() < 0.018


def test_oracle_verification_edges():
    p = np.array([[0.5, 0.5, 0.0], [0.0, 0.0, 1.0]])
    assert S.verify_tree(p, p, np.array([0, 1]), [-1, 0], np.array([0.3, 0.999])) == ([0, 1], 2)
    assert S.verify_tree(p, None, np.array([0, 2]), [-1, 0], np.array([0.6, 0.0])) == ([0], 1)   # p(2) = 0
    assert S.verify_tree(p, None, np.array([0, 7]), [-1, 0], np.array([0.0, 0.0])) == ([0], 0)   # no such token
    assert S.verify_tree(0 * p, p, np.array([0, 1]), [-1, 0], np.array([0.0, 0.0])) == ([0], -1)
