"""How the library cuts the block operators' calls up, worked out from the workspaces it asks for."""
import test_sequence_layers_amd as T


def _up(n):
    return (n + 255) // 256 * 256


def scan_segments(B, N, C, S, G=1, backward=False, dtype=T.TTT_BF16):
    """(segments of a sequence, at most this many tokens each): of the forward pass the end states [S][C] and a sum
    [C] of each; of the backward pass two such states, a sum, and partial sums [S + 2][C] of each, beside checkpoints
    ([S + 1][C]) every 8 tokens and the channel blocks' sums [2 S] of every token. The forward plan is that with or
    without lengths which has more segments."""
    lib = T.load_library()
    if not backward:
        need = lib.ttt_forward_selective_scan_workspace(dtype, B, N, C, S, G)
        nseg = max(1, need // (4 * B * (S + 1) * C))
    else:
        need = lib.ttt_backward_selective_scan_workspace(dtype, B, N, C, S, G)
        blocks, subs = (C // G + 63) // 64 * G, (N + 7) // 8
        rest = _up(4 * B * subs * S * C) + _up(4 * B * subs * C) + _up(4 * B * N * blocks * 2 * S)
        fits = [n for n in range(1, (N + 7) // 8 + 1)
                if 2 * _up(4 * B * n * S * C) + _up(4 * B * n * C) + _up(4 * B * n * (S * C + 2 * C)) + rest == need]
        assert len(fits) >= 1, need
        nseg = fits[0]
    return nseg, -(-N // nseg)
