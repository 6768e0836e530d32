"""decode_attn_paged's checks in Python (no GPU is needed: the device is compared last)."""
import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    import rank_compressed_kv_b200 as kv
    return kv


def _args(kv):
    """Arguments that only their device speaks against."""
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    return dict(dims=kv.Dims(batch=3, n_q_heads=16, n_kv_heads=8, T_vis=100, L_text_cap=0),
                pdims=kv.PagedDims(batch=3, n_q_heads=16, n_kv_heads=8, page_size=64, n_pages=10, max_pages=5), n_layers=2,
                q=z(6, 16, 128), CK_lo=z(12, 100, 16), CK_hi=z(12, 100, 48), BK=z(12, 64, 512), CV_lo=z(12, 100, 16),
                CV_hi=z(12, 100, 48), BV=z(12, 64, 512), K_pages=z(2, 10, 8, 64, 128), V_pages=z(2, 10, 8, 64, 128),
                block_table=torch.zeros(3, 5, dtype=torch.int32), seq_lens=torch.zeros(3, dtype=torch.int32),
                mask=torch.zeros(12, 4, dtype=torch.int32), scale=1.0, out=z(6, 16, 128), mass=torch.zeros(12, 100),
                ws=torch.zeros(100, dtype=torch.uint8))


def test_it_refuses_tensors_that_are_not_on_the_current_device(kv):
    with pytest.raises(ValueError, match="K_pages is not on the current CUDA device"):
        kv.decode_attn_paged(**_args(kv))


@pytest.mark.parametrize("over,text", [
    (dict(block_table=torch.zeros(5, 3, dtype=torch.int32)), "block_table has shape"),
    (dict(block_table=torch.zeros(15, dtype=torch.int32)), "block_table has shape"),
    (dict(block_table=torch.zeros(3, 6, dtype=torch.int32)), "block_table has shape"),
    (dict(block_table=torch.zeros(5, 3, dtype=torch.int32).T), "contiguous"),
    (dict(block_table=torch.zeros(3, 5, dtype=torch.int64)), "block_table is torch.int64"),
    (dict(seq_lens=torch.zeros(3, 1, dtype=torch.int32)), "seq_lens has shape"),
    (dict(seq_lens=torch.zeros(4, dtype=torch.int32)), "seq_lens has shape"),
    (dict(seq_lens=torch.zeros(6, dtype=torch.int32)[::2]), "contiguous"),
    (dict(seq_lens=torch.zeros(3)), "seq_lens is torch.float32"),
    (dict(K_pages=torch.zeros(2, 9, 8, 64, 128, dtype=BF)), "K_pages has shape"),
    (dict(V_pages=torch.zeros(1, 10, 8, 64, 128, dtype=BF)), "V_pages has shape"),
    (dict(V_pages=torch.zeros(2, 10, 8, 64, 128, dtype=torch.float16)), "V_pages is torch.float16"),
    (dict(K_pages=torch.zeros(2, 10, 8, 128, 64, dtype=BF).transpose(3, 4)), "contiguous"),
])
def test_it_refuses(kv, over, text):
    with pytest.raises(ValueError, match=text):
        kv.decode_attn_paged(**{**_args(kv), **over})


def test_other_objects_are_not_tensors(kv):
    for name in ("block_table", "seq_lens", "K_pages", "V_pages"):
        with pytest.raises(TypeError, match=f"{name} is not a tensor"):
            kv.decode_attn_paged(**{**_args(kv), name: None})


def test_pools_whose_size_passes_64_bits(kv):
    """8193 layers of 67100673 pages of 2^25 elements: 2^64 + 2^25, which is not 2^25."""
    d = kv.PagedDims(batch=1, n_q_heads=1024, n_kv_heads=1024, page_size=256, n_pages=67100673, max_pages=1)
    assert 8193 * d.n_pages * 2 ** 25 == 2 ** 64 + 2 ** 25
    k = torch.zeros(1, 1, 1024, 128, dtype=BF).expand(8193, 1, 1024, 128)
    pool = torch.empty(2 ** 25, dtype=BF)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="K_pages has shape"):
        kv.paged_append(d, 8193, None, None, None, None, k, k, None, i, i[None], None, pool, pool)
