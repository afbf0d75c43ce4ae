"""CPU test of the norm's workspace: the bound that its workgroups' column sums keep (no call below reaches a GPU)."""
import gated_mlp_gemms_amd as gm


def test_column_sums_are_bounded():
    """With rows enough for any number of workgroups: 25 MiB up to widths of 6144, and 256 workgroups' two fp32 sums a column
    from there to the widest rows that are held in registers (fp32 8192, 16-bit 16384: 32 MiB)."""
    for d in range(8, 16385, 8):
        b = gm.norm_workspace_bytes(1 << 20, d)
        assert b <= (25 << 20 if d <= 6144 else 256 * 2 * d * 4), d
