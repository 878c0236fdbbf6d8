"""Products for the forms of mhc_linear: (mxfp8, gated) to rows, in features, out features
and the form the library takes, (pairs of CTAs, CTAs that divide a tile's K, CTAs per SM).
Together with the products of test_linear_every_form they reach every form there is."""

MORE_FORMS = {
    (False, False): [(2, 976, 1, (False, 4, 1)), (2, 1744, 1, (False, 6, 1)), (35, 1744, 129, (False, 6, 1))],
    (False, True): [(2, 8, 1, (False, 1, 1)), (692, 1288, 1, (False, 3, 1)), (2, 792, 1, (False, 5, 1))],
    (True, False): [(2, 1184, 1, (False, 2, 1)), (3, 1184, 9501, (False, 2, 2)), (3, 1312, 5853, (False, 3, 2)),
                    (2, 1952, 4359, (False, 4, 2)), (2, 2624, 1, (False, 5, 1)), (2, 2784, 3437, (False, 5, 2)),
                    (2, 3296, 2927, (False, 6, 2))],
    (True, True): [(3, 1696, 8960, (False, 2, 1)), (2, 2464, 11904, (False, 2, 2)), (5, 2624, 5632, (False, 3, 1)),
                   (3, 1440, 8320, (False, 3, 2)), (2, 1312, 4352, (False, 4, 2)), (2, 1568, 128, (False, 5, 1)),
                   (2, 1600, 3456, (False, 5, 2)), (2, 2016, 2944, (False, 6, 2))],
}
