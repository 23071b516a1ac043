"""Which form of the product kernel a call takes: the host's rules, restated so that a test can say which form it runs.

"cluster": the blocks of a cluster share a tile's K (few tiles); "pairs": two blocks a tile of 256 rows; "one": a block a tile."""
import torch

SPLITS = ((8, 4, 66), (6, 8, 66), (5, 8, 66), (4, 2, 100), (3, 2, 80), (2, 2, 100))   # blocks, blocks of K each, % of the SMs


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def form_of(rows, groups, N, K, expected=0, offsets=True):
    """rows: what the arrays hold (regions: groups * cap, offsets=False)."""
    tiles = min((rows + groups * 127) // 128, rows) * -(-N // 256)
    for split, blocks, percent in SPLITS:
        if K // 128 >= split * blocks and tiles * split * 100 <= sms() * percent:
            return "cluster"
    per = expected or rows // groups // (16 if groups > 1 and not offsets else 1)
    return "pairs" if per > 128 and (per <= 256 or per > 384) else "one"


def tiles_of(counts, N, form):
    """(tiles of the groups, blocks or pairs that share them)."""
    rows, units = (256, sms() // 2) if form == "pairs" else (128, sms())
    return sum(-(-c // rows) for c in counts) * -(-N // 256), units
