"""Calls that the binding of the speculative step refuses before it launches
anything: shapes, types, devices and layouts that do not fit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_kv_continuous_gb300 import ops as o
    return o


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def f32(*shape):
    return torch.zeros(shape, device="cuda")


def refuses(ops, fn, good, **bad):
    with pytest.raises(ops.PagedAttentionError):
        fn(**{**good, **bad})


def test_decode_tree(ops):
    good = dict(q=bf16(4, 4, 128), cu_seqlens=i32(3), parents=i32(4), k_cache=bf16(3, 16, 2, 128),
                v_cache=bf16(3, 16, 2, 128), block_tables=i32(2, 1), context_lens=i32(2),
                scale=0.1, max_q_len=4)
    assert ops.decode_tree(**good).shape == (4, 4, 128)
    for bad in (dict(q=f32(4, 4, 128)), dict(q=bf16(4, 4, 64)), dict(q=bf16(4, 8, 128)[:, ::2]),
                dict(parents=i32(3)), dict(parents=i32(4).long()), dict(cu_seqlens=i32(0)),
                dict(k_cache=bf16(3, 16, 2, 64)), dict(v_cache=bf16(2, 16, 2, 128)),
                dict(block_tables=i32(1, 1)), dict(context_lens=i32(3)),
                dict(block_tables=i32(2, 4)[:, ::2]), dict(out=bf16(4, 4, 64)),
                dict(out_dtype=torch.float16), dict(parents=i32(4).cpu()),
                dict(max_q_len=-1), dict(scale=float("nan")), dict(num_splits=5000),
                dict(workspace=i32(64)), dict(k_cache=bf16(3, 16, 3, 128),
                                              v_cache=bf16(3, 16, 3, 128))):
        refuses(ops, ops.decode_tree, good, **bad)


def test_verify_tree(ops):
    good = dict(tokens=i32(4), parents=i32(4), cu_seqlens=i32(3), target_probs=f32(4, 9),
                uniforms=f32(4), sample_uniforms=f32(2), max_q_len=4, draft_probs=f32(4, 9))
    assert [tuple(t.shape) for t in ops.verify_tree(**good)] == [(2,), (2, 4), (2, 4)]
    for bad in (dict(tokens=i32(3)), dict(parents=i32(5)), dict(target_probs=f32(3, 9)),
                dict(target_probs=bf16(4, 9)), dict(draft_probs=f32(4, 8)),
                dict(target_probs=f32(9, 4).t()), dict(draft_probs=f32(1, 9).expand(4, 9)),
                dict(uniforms=f32(4).double()), dict(sample_uniforms=f32(3)),
                dict(max_q_len=-1), dict(path=i32(2, 3)), dict(accepted=i32(3)),
                dict(out_tokens=i32(2, 8)[:, ::2]), dict(error_flags=i32(0)),
                dict(uniforms=f32(4).cpu())):
        refuses(ops, ops.verify_tree, good, **bad)


def test_commit_tree(ops):
    pools = ops.PagePools([bf16(3, 16, 2, 128)])
    good = dict(pools=pools, cu_seqlens=i32(3), block_tables=i32(2, 1), context_lens=i32(2),
                path=i32(2, 4), accepted=i32(2), ref_counts=i32(3))
    ops.commit_tree(**good)
    for bad in (dict(path=i32(1, 4)), dict(accepted=i32(3)), dict(ref_counts=i32(2)),
                dict(context_lens=i32(3)), dict(path=i32(2, 8)[:, ::2]),
                dict(block_tables=i32(1, 1)), dict(cu_seqlens=i32(0)),
                dict(pools=ops.PagePools([bf16(3, 2, 128, 8)])),  # (a dim-major pool)
                dict(pools=ops.PagePools([i32(3)])), dict(path=i32(2, 4).long())):
        refuses(ops, ops.commit_tree, good, **bad)


def test_nothing_to_do(ops):
    """No sequences, no rows: nothing is launched, and the outputs are empty."""
    out = ops.decode_tree(bf16(0, 4, 128), i32(1), i32(0), bf16(3, 16, 2, 128),
                          bf16(3, 16, 2, 128), i32(0, 1), i32(0), 0.1, 0)
    assert out.shape == (0, 4, 128)
    got = ops.verify_tree(i32(0), i32(0), i32(1), f32(0, 9), f32(0), f32(0), 4)
    assert [tuple(t.shape) for t in got] == [(0,), (0, 4), (0, 4)]
    ops.commit_tree(ops.PagePools([bf16(3, 16, 2, 128)]), i32(1), i32(0, 1), i32(0), i32(0, 4),
                    i32(0))
    torch.cuda.synchronize()
