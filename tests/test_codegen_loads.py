"""The projections' loads in the generated code (CPU only): what the hardware checks against a buffer's end."""
import re

from test_codegen import disassembly  # noqa: F401  (the library's device code)


def scale_loads(text):
    """{kernel: (tiles of 16 tokens, [(vector offset, scalar offset) of each load of a scale byte])}"""
    found, at = {}, None
    for line in text.split("\n"):
        m = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if m:
            rows = re.search(r"project_rows_kernelILi\d+ELb[01]ELi(\d+)ELi\d+EE", m.group(1))
            at = found.setdefault(m.group(1), (int(rows.group(1)), [])) if rows else None
        elif at is not None and line.strip().startswith("buffer_load_ubyte"):
            v = re.match(r"\s*buffer_load_ubyte v\d+, (v\d+), s\[\d+:\d+\], (\S+) offen(?:\s|$)", line)
            assert v, line
            at[1].append(v.groups())
    return found


def test_rows_of_scales_are_in_the_checked_offset(disassembly):  # noqa: F811
    """A load past the last token's scales gives zeros only by its vector offset: a scalar offset is not part of the check
    against the buffer's end.  Each step loads a byte for every 16 tokens, with one scalar offset (the group) and rows of
    its own in the vector offset."""
    found = scale_loads(disassembly)
    assert {tiles for tiles, _ in found.values()} == {1, 2, 4}
    for name, (tiles, loads) in found.items():
        assert loads and len(loads) % tiles == 0, name
        for i in range(0, len(loads), tiles):
            step = loads[i:i + tiles]
            assert len({scalar for _, scalar in step}) == 1 and len({rows for rows, _ in step}) == tiles, (name, step)


def test_value_rows_of_a_prefill_are_in_the_checked_offset(disassembly):  # noqa: F811
    """The scan's rows of v end at the sequence's last token: the loads of a chunk's rows, those before its gates' load
    from the same buffer, have no scalar offset."""
    kernels, loads = {}, None
    for line in disassembly.split("\n"):
        m = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if m:
            loads = kernels.setdefault(m.group(1), []) if "prefill_scan_kernel" in m.group(1) else None
        elif loads is not None:
            m = re.match(r"\s*(buffer_load_dword\S*) v\d+, (s\[\d+:\d+\]), (\S+) offen.* lds", line)
            if m:
                loads.append(m.groups())
    assert kernels
    for name, loads in kernels.items():
        gates = [i for i, x in enumerate(loads) if x[0] == "buffer_load_dword"]
        assert gates, name
        for i in gates:
            rows = loads[i - 1][1]
            j = i - 1
            while j >= 0 and loads[j][:2] == ("buffer_load_dwordx4", rows):
                assert loads[j][2] == "0", (name, loads[j])
                j -= 1
            assert i - 1 - j >= 2, name
