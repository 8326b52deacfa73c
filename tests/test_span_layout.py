"""How the span attentions lay out their work, as their workspace queries show it (no GPU)."""

import pytest

from test_span_args import D, lib, tree, window  # noqa: F401


@pytest.mark.parametrize("B,T,H,longest", [(32, 256, 16, 8), (8, 322, 128, 48), (16, 16, 128, 1), (40, 90, 24, 5),
                                           (3, 500, 3, 200)])
def test_loose_max_q_changes_nothing(lib, B, T, H, longest):  # noqa: F811
    """What decides the split is the query rows that there can be, not B times the longest sequence that max_q allows:
    leaving max_q at T (always enough) splits long contexts, and leaves windows whole, as the exact value does."""
    for max_q in (T, 10 * T):
        for ctx in (16384, 100000):
            assert (lib.ls_tree_attention_workspace_size(B, T, H, longest, 1 << 20, ctx, 0, 1, 0) > 0) == \
                (lib.ls_tree_attention_workspace_size(B, T, H, max_q, 1 << 20, ctx, 0, 1, 0) > 0)
        assert (lib.ls_window_attention_workspace_size(B, T, H, longest, 512, 1, 4) > 0) == \
            (lib.ls_window_attention_workspace_size(B, T, H, max_q, 512, 1, 4) > 0)


def test_many_padded_sequences_are_taken(lib):  # noqa: F811
    """Two million sequences, most without tokens, max_q at its default: the call gets as far as its workspace."""
    B, T = 1 << 21, 600
    assert lib.ls_tree_attention_workspace_size(B, T, 128, T, 1 << 20, 100000, 0, 1, 0) > 0
    assert tree(lib, B=B, T=T, H=128, max_q=T, n=1 << 20, max_ctx=100000) == 2
    assert window(lib, B=(1 << 24) + 1) == 1
    assert lib.ls_window_attention_workspace_size((1 << 24) + 1, 4, 16, 4, 64, 1, 4) == 0


def test_sinks_up_to_the_largest_int(lib):  # noqa: F811
    """n_sink may say "all": the number of its tiles is formed in 64 bits."""
    big = (1 << 31) - 1
    size = lambda n: lib.ls_window_attention_workspace_size(1, 3, 16, 3, 512, 1, n)  # noqa: E731
    assert size(big) == size(big - 500) == size(1 << 24) > 0
    assert window(lib, sink=big) == 2 and window(lib, sink=big - 500) == 2


def test_short_windows_stay_whole(lib):  # noqa: F811
    """Fewer query tiles than pairs with a few tiles each are dealt out whole, with one launch and no workspace."""
    for B, n, H in ((32, 8, 16), (1, 30, 128), (40, 1, 128), (64, 1, 128)):
        assert lib.ls_window_attention_workspace_size(B, B * n, H, n, 512, 1, 4) == 0
