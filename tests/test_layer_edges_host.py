"""The SSD layer's serving operators on the CPU: how packed sequences are cut, and what the binding decides before a launch."""
import selective_state_space_55_amd as mscan


def test_ssd_a_long_sequence_among_short_ones_is_cut_without_a_hint():
    f = mscan.ssd_fwd_varlen_workspace_size
    shape = (64, 64, 128)   # 32 workgroups a piece
    # one of 58000, 50000 or 30000 tokens may be among these; the mean, two to four pieces, does not tell
    for nseq, total in ((20, 60000), (28, 60000), (16, 32768), (16, 65536), (20, 12000), (16, 4096)):
        assert f(nseq, total, *shape) > 0, (nseq, total)
    # with the longest sequence known, those that fill the GPU by themselves stay whole up to four pieces
    assert f(16, 4096, *shape, 1, 256) == 0 and f(20, 60000, *shape, 1, 4096) == 0
    assert f(20, 60000, *shape, 1, 58000) > 0
