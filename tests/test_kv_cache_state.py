"""omq.KVCache's state on the CPU: what it refuses to be made of."""
import pytest


@pytest.fixture(scope="module")
def omq():
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


@pytest.mark.parametrize("max_len,page,n_pos", [(100, 64, 100), (100, 64, 127), (128, 64, 64), (1, 16, 15)])
def test_rotary_tables_shorter_than_the_block_table_are_refused(omq, max_len, page, n_pos):
    """The plan grants whole pages: 100 tokens in pages of 64 have positions up to 127."""
    with pytest.raises(ValueError, match="n_pos"):
        omq.KVCache(1, 4, 1, 64, page=page, max_len=max_len, n_pos=n_pos, device="cpu")


@pytest.mark.parametrize("max_len,page,n_pos,want", [(100, 64, None, 128), (100, 64, 128, 128), (128, 64, None, 128),
                                                     (33, 48, 500, 500), (1, 16, None, 16)])
def test_rotary_table_covers_every_position_of_the_block_table(omq, monkeypatch, max_len, page, n_pos, want):
    made = []
    monkeypatch.setattr(omq, "rope_table", lambda n, D, base, device: made.append(n))
    cache = omq.KVCache(1, 4, 1, 64, page=page, max_len=max_len, n_pos=n_pos, device="cpu")
    assert made == [want] and want >= cache.table.shape[1] * page
