"""How the convolution and the scan's backward pass cut their work, restated from the rules in csrc/conv.cu and
csrc/scan_bwd.cu, so that a test can say which of their paths its sizes reach. The workspace sizes that the library
gives follow from the same numbers, which ties the restatement to it."""
import ctypes


def ceil(a, b):
    return -(-a // b)


def conv_run(B, H, T, d, V, slots):
    """(tokens of a thread's run, blocks along the tokens) with V channels a thread and `slots` resident blocks."""
    packs = H * ceil(d, V)
    bx = 32
    while bx < 256 and bx < packs:
        bx *= 2
    by = 256 // bx
    rows = ceil(packs, bx) * max(B, 1)
    for turns in range(1, 9):
        tiles = slots * turns // rows if slots * turns > rows else 1
        run = ceil(T, tiles * by)
        if run <= 160:
            break
    run = min(max(run, 8), 160)
    return run, max(ceil(T, run * by), 1)


def conv_fwd_run(B, H, T, d, K, V, sms):
    return conv_run(B, H, T, d, V, sms * (4 if K <= 4 else 2))[0]


def conv_bwd_run(B, H, T, d, K, V):
    return conv_run(B, H, T, d, V, 148 * (3 if K <= 4 else 2))[0]


def conv_workspace(B, H, T, d, K):
    return max(B * conv_run(B, H, T, d, V, 148 * (3 if K <= 4 else 2))[1] * H * d * (K + 1) * 4 for V in (1, 2))


class ScanBwd:
    """nseg segments of 16 tokens, `walk` of them a walk, nwalk walks, `block` walks a block of the first step."""

    def __init__(self, B, H, T, dk, dv):
        lanes = 1
        while lanes * 4 < dk:
            lanes *= 2
        channels = 32 // lanes * 4 * (1 if lanes == 1 else 2 if lanes == 2 else 4)
        self.ngrp = ceil(dv, channels)
        self.cols = max(c for c in (4, 8, 16, 32, 64, 128) if c == 4 or c < 2 * dk)
        self.nseg = ceil(T, 16)
        turns = lambda blocks: ceil(blocks, 148 * 3)
        best = None
        for walk in range(1, 33):
            n = ceil(self.nseg, walk)
            cost = turns(self.ngrp * B * H * n) * (walk * 16 + 4) + 0.4 * n
            if best is None or cost < best:
                best, self.walk = cost, walk
        self.nwalk = ceil(self.nseg, self.walk)
        groups = B * H * ceil(dv, 128 // (1 if dk <= 16 else 2 if dk <= 32 else 4 if dk <= 64 else 8))
        best = None
        for n in range(1, 17):
            cost = turns(groups * ceil(self.nwalk, n)) * (n * self.walk * 16 + 24)
            if best is None or cost < best:
                best, self.block = cost, n
        rows = B * H * dv
        self.bytes = 4 * (rows * (self.nseg * (self.cols + 1) + self.nwalk * (2 * self.cols + 1 + dk + 2))
                          + (2 * self.ngrp * B * H * T * dk if self.ngrp > 1 else 0))


def size(L, name, args):
    return getattr(L, f"falcon_{name}_bwd_workspace_size")(ctypes.byref(args))
