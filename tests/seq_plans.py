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


# Scans that between them take every branch of the library's plans: B, N, C, S, G, dtype, options, and the tokens of a
# segment that they have at least (forward; N: in one launch), (backward).
SCAN_CASES = [
    (2, 4096, 768, 16, 1, "bf16", dict(), 32, 32),                          # three waves per SIMD; four sub-chunks
    (4, 8192, 768, 16, 1, "bf16", dict(), 64, 128),                         # six; sixteen
    (3, 1999, 1000, 32, 2, "fp32", dict(lengths=[1999, 777, 1500]), 24, 56),  # wide states, lengths
    (1, 1024, 768, 16, 1, "bf16", dict(gate=False), 12, 16),                # by the root of the length
    (2, 2048, 256, 16, 256, "fp32", dict(lengths=[2048, 1111]), 200, 300),  # a group for each channel: long segments
    (1, 6000, 300, 8, 150, "fp32", dict(), 150, 300),
    (2, 1500, 320, 64, 320, "bf16", dict(), 180, 700),
    (1, 3000, 1600, 32, 1600, "fp32", dict(gate=False), 3000, 1500),        # one launch by blocks; no more than 2048
    (4, 700, 410, 8, 410, "bf16", dict(lengths=[700, 0, 699, 300]), 700, 350),
    (2, 600, 650, 16, 650, "fp32", dict(), 600, 200),
    (1, 400, 830, 64, 830, "fp32", dict(), 400, 400),                       # one segment backward
    (2, 100, 200, 16, 200, "bf16", dict(sp=False), 100, 15),                # one launch by length
]
# Layer norms whose backward pass walks at least three turns, the last one ragged: M, H, D, dtype, sliced, and the tokens
# that all workgroups take at a time.
NORM_CASES = [
    (12544, 1, 384, "bf16", False, 16 * 256), (40000, 12, 64, "bf16", True, 10 * 256), (20001, 5, 16, "fp32", False, 25 * 256),
    (1700, 1, 2056, "bf16", False, 512), (1700, 1, 4096, "fp32", False, 512), (1100, 1, 8192, "bf16", False, 256),
    (600, 1, 16384, "bf16", False, 256), (700, 1, 16384, "fp32", False, 256), (5001, 1, 1001, "fp32", False, 4 * 512),
    (9001, 1, 100, "bf16", False, 16 * 256), (9001, 1, 33, "fp32", False, 16 * 256), (1101, 1, 2050, "fp32", False, 512),
    (600, 1, 5001, "bf16", False, 256), (601, 1, 8193, "fp32", False, 256), (401, 300, 8, "fp32", False, 85),
    (5003, 1, 768, "bf16", True, 4 * 512), (4901, 1, 768, "fp32", False, 4 * 512),
]
CONV_CASES = [  # B, N, C, K, dtype, silu, state, lengths
    (4, 8192, 768, 4, "bf16", True, False, None), (2, 5000, 193, 3, "fp32", False, True, [5000, 1234]),
    (3, 1000, 260, 2, "fp32", True, True, None), (1, 16384, 64, 4, "fp32", True, True, None), (5, 300, 66, 4, "bf16", True, True, [300, 0, 2, 64, 299]),
]
