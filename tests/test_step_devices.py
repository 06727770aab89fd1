"""The binding of the calls around the indexer lets no tensor through that the GPU cannot read."""

import pytest
import torch


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_nvfp4_gb300 import build

    build.build()
    import sparse_attention_indexer_nvfp4_gb300 as idx

    return idx


def calls(idx, device):
    """Each function with arguments that pass every check but, perhaps, that of the device."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64, device=device)
    f32 = lambda *s: torch.zeros(s, device=device)
    half = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=device)
    size = idx.idx_tree_attention_workspace_bytes(1, 2, 4, 2, 64, 2, 4)
    return {
        idx.idx_build_slots: dict(ctx_lens=i32(2), new_lens=i32(2), owned_pages=i32(2), block_table=i32(2, 3), free_blocks=i32(4),
                                  free_cursor=i32(1), num_blocks=9, page_tokens=4, cu_tokens=i32(3), seq_lens=i32(2), pages_out=i32(2),
                                  cursor_out=i32(1), positions=i32(6), slots=i64(6), parents=i32(6), tree_mask=i64(6), status=i32(1)),
        idx.idx_rope_append: dict(q=f32(5, 2, 8), k=f32(5, 2, 8), v=f32(5, 2, 8), positions=i32(5), slots=i64(5), q_out=f32(5, 2, 8),
                                  inv_freq=torch.zeros(4, dtype=torch.float64, device=device), k_cache=f32(2, 4, 2, 8),
                                  v_cache=f32(2, 4, 2, 8), status=i32(1)),
        idx.idx_tree_attention: dict(q=half(2, 4, 64), k_cache=half(3, 16, 2, 64), v_cache=half(3, 16, 2, 64), block_table=i32(1, 2),
                                     seq_lens=i32(1), cu_tokens=i32(2), out=half(2, 4, 64), scale=1.0, tree_mask=i64(2),
                                     pages=i32(1, 2, 2, 4), lse=f32(2, 4), status=i32(1),
                                     workspace=torch.zeros(size, dtype=torch.uint8, device=device)),
        idx.idx_verify_drafts: dict(target=f32(4, 9), draft=f32(4, 9), tokens=i32(4), cu_tokens=i32(2), accept_u=f32(4), sample_u=f32(1),
                                    out_tokens=i32(1, 3), out_nodes=i32(1, 3), num_accepted=i32(1), parents=i32(4), status=i32(1)),
    }


def test_host_tensors_are_refused(idx):
    for fn, args in calls(idx, "cpu").items():
        with pytest.raises(ValueError, match="is on cpu"):
            fn(**args, stream=1)


def test_status_is_checked(idx):
    for fn, args in calls(idx, "cpu").items():
        for bad, what in ((torch.zeros(1), "status has type"), (torch.zeros(1, dtype=torch.int64), "status has type"),
                          (torch.zeros(0, dtype=torch.int32), "status has no element")):
            with pytest.raises(ValueError, match=what):
                fn(**(args | dict(status=bad)), stream=1)


@pytest.mark.gpu
def test_one_host_tensor_is_refused_by_name(idx):
    """Among tensors of the GPU: answered before anything is launched."""
    for fn, args in calls(idx, "cuda").items():
        for name, t in args.items():
            if torch.is_tensor(t):
                with pytest.raises(ValueError, match=f"{name} is on cpu"):
                    fn(**(args | {name: t.cpu()}))


@pytest.mark.gpu
def test_tensors_of_the_gpu_pass(idx):
    for fn, args in calls(idx, "cuda").items():
        assert fn(**args) == 0
        assert fn(**(args | dict(status=None))) == 0
    torch.cuda.synchronize()
