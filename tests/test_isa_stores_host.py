"""Wide buffer stores in the library's device code (built here; no GPU needed).

A store of more than 8 bytes reads its data registers a state after it is issued. Where it has no scalar offset the compiler
keeps a vector instruction that writes them one state behind; with a scalar offset it does not, and on gfx950 such stores
have taken the registers' new contents. So the code holds none.
"""
import re

from tests.test_isa_host import listings, pytestmark  # noqa: F401

STORE = re.compile(r"buffer_store_dwordx[34] v\[\d+:\d+\], \S+, s\[\d+:\d+\], (\S+)")


def test_the_pattern_tells_offsets_apart():
    assert STORE.match("buffer_store_dwordx4 v[66:69], v70, s[8:11], s2 offen nt").group(1) == "s2"
    assert STORE.match("buffer_store_dwordx4 v[66:69], v70, s[8:11], 0 offen nt").group(1) == "0"


def test_wide_buffer_stores_have_no_scalar_offset(listings):  # noqa: F811
    found = 0
    for lines in listings:
        for ins in lines:
            m = STORE.match(ins)
            if m:
                found += 1
                assert not m.group(1).startswith(("s", "m0", "vcc", "ttmp")), ins
    assert found
