"""The decoding attention's deal of its work to teams and CTAs (csrc/usp_paged.cuh), on the host."""
import platform

from test_paged_rows import build_and_run


def test_every_tile_once_and_every_part_found(tmp_path):
    # (on 64-bit Arm the address sanitizer hangs at its start where the kernel spreads addresses over more bits than it knows)
    build_and_run("paged_deal", tmp_path, "address,undefined" if platform.machine() == "x86_64" else "undefined")
