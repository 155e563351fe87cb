"""What the header says of dsa_latent_attn_shared's workspace is what the library asks for (no device is
touched)."""
import pytest


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_index_gb300 as m
    return m


@pytest.mark.parametrize("B,Sq,H,G", [
    (1, 1, 1, 1), (3, 1, 16, 1), (8, 1, 16, 1), (64, 1, 16, 1), (64, 1, 16, 64), (1024, 1, 8, 4), (4096, 1, 1, 1),
    (4096, 1, 8, 64), (31, 5, 3, 2), (7, 200, 128, 5), (1, 4096, 128, 1)])
def test_documented_size(dsa, B, Sq, H, G):
    """Few heads and many sequences among them, where a sequence's part has more rows than it uses."""
    rows = B * Sq * H
    parts = rows // 128 + min(G, B) + B * -(-Sq * H // 128) + 80
    fp32 = parts * min(128, -(-rows // 32) * 32) * 2056
    # 8 bytes a tile, and the groups' starts and tiles
    assert fp32 <= dsa.latent_attn_shared_workspace_bytes(B, Sq, H, G, 512, 64) <= fp32 + 8 * parts + 1024


def test_documented_examples(dsa):
    for (B, H), size in {(64, 16): 40.3e6, (1024, 8): 308e6, (4096, 1): 1.1e9}.items():
        got = dsa.latent_attn_shared_workspace_bytes(B, 1, H, 1, 512, 64)
        assert 0.97 * size <= got <= 1.03 * size, (B, H, got)
