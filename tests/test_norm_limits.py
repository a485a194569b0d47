"""Which lists the gradient norm takes in one launch (no workspace), at the
limit of 128 tiles of 64 16-byte blocks, counted as if every tensor started on
the last byte of a 128-byte line.  No GPU call is made."""
import ctypes

import pytest

import fsdp_sharded_state_amd as fs

TILES = 128
# Most elements of a tensor of t tiles: t * 64 blocks hold its bytes, the 127
# before them and less than one block after: 1024 t >= 127 + bytes, rounded up to 16.
MOST = {fs.FS_BF16: lambda t: (1024 * t - 127) // 2, fs.FS_FP32: lambda t: (1024 * t - 127) // 4}


def workspace(numels, codes) -> int:
    n, need = len(numels), ctypes.c_int64(-1)
    rc = fs.lib().fs_grad_norm_workspace(n, (ctypes.c_int64 * max(1, n))(*numels), (ctypes.c_int32 * max(1, n))(*codes),
                                         ctypes.byref(need))
    assert rc == 0
    return need.value


@pytest.mark.parametrize("code", [fs.FS_BF16, fs.FS_FP32])
def test_one_launch_up_to_128_tiles(code):
    most = MOST[code]
    assert workspace([most(TILES)], [code]) == 0
    assert workspace([most(TILES) + 1], [code]) > 0
    # one tile each, empty tensors aside
    assert workspace([most(1)] * TILES + [0] * 300, [code] * (TILES + 300)) == 0
    assert workspace([most(1)] * (TILES + 1), [code] * (TILES + 1)) > 0
    assert workspace([1] * TILES, [code] * TILES) == 0
    assert workspace([1] * (TILES + 1), [code] * (TILES + 1)) > 0
    # two of 64 tiles, and one element more
    assert workspace([most(64)] * 2, [code] * 2) == 0
    assert workspace([most(64), most(64) + 1], [code] * 2) > 0


def test_mixed_types_count_together():
    numels = [MOST[fs.FS_BF16](100), MOST[fs.FS_FP32](28)]
    codes = [fs.FS_BF16, fs.FS_FP32]
    assert workspace(numels, codes) == 0
    assert workspace(numels + [1], codes + [fs.FS_BF16]) > 0
